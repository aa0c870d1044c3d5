"""Views of outputs that rc_kv_attend refuses, and views that it takes, without a GPU:
every call here is refused, for its output's view or else for an lse out of alignment."""
import pytest
import torch

SIZES = dict(batch=3, q_heads=4, kv_heads=2, head_dim=64, pool_blocks=12, seq_blocks=4, max_queries=5)
A = 4096


@pytest.fixture(scope="module")
def rc():
    from activation_residual_compression_amd import librescomp
    return librescomp


def status(rc, plan, strides, queries=5):
    q = rc.rc_kv_view_t(A, rc.RC_BF16, 5 * 4 * 64, 4 * 64, 64)
    try:
        rc.rc_kv_attend(plan.handle, 0, rc.rc_kv_cache_t(A, A, A, A, A, A), None, A, 0, queries, q, None,
                        rc.rc_kv_view_t(A, rc.RC_BF16, *strides), A + 2)
    except rc.RcError as e:
        return e.status
    return rc.RC_OK


@pytest.mark.parametrize("strides", [
    (64, 64, 64),                                  # all the same
    (20 * 64, 64, 64),                             # tokens over heads
    (4 * 64, 4 * 64, 64),                          # sequences over tokens
    (19 * 64, 4 * 64, 64),                         # the next sequence begins in the last token
    (20 * 64, 3 * 64, 64),                         # the next token begins in the last head
    (64, 3 * 64, 14 * 64),                         # sequences inside, heads outside, one row short
])
def test_outputs_that_overlap_are_refused(rc, strides):
    with rc.KvPlan(**SIZES) as plan:
        assert status(rc, plan, strides) == rc.RC_ERR_INVALID_ARG


@pytest.mark.parametrize("shape,order,cut", [
    ((3, 5, 4, 64), (0, 1, 2), None), ((5, 3, 4, 64), (1, 0, 2), None), ((4, 3, 5, 64), (1, 2, 0), None),
    ((4, 5, 3, 64), (2, 1, 0), None), ((3, 4, 5, 64), (0, 2, 1), None), ((5, 4, 3, 64), (2, 0, 1), None),
    ((3, 9, 7, 64), (0, 1, 2), (slice(None), slice(2, 7), slice(1, 5))),
    ((6, 5, 8, 64), (0, 1, 2), (slice(0, 6, 2), slice(None), slice(0, 8, 2)))])
def test_outputs_that_are_views_of_a_tensor_are_taken(rc, shape, order, cut):
    x = torch.empty(shape, dtype=torch.bfloat16)
    x = (x[cut] if cut else x).permute(*order, 3)
    assert x.shape == (3, 5, 4, 64)
    with rc.KvPlan(**SIZES) as plan:
        assert status(rc, plan, x.stride()[:3]) == rc.RC_ERR_ALIGNMENT


def test_dimensions_of_one_do_not_count(rc):
    with rc.KvPlan(**{**SIZES, "batch": 1}) as plan:
        assert status(rc, plan, (0, 4 * 64, 64)) == rc.RC_ERR_ALIGNMENT
        assert status(rc, plan, (0, 0, 64), queries=1) == rc.RC_ERR_ALIGNMENT
