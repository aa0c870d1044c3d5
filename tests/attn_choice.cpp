// The host's choice for a call of attention over packed sequences, without a GPU: the plan's code as it is, with
// memory that nothing reads and launches that only write down what they were given.
#include "../activation_residual_compression_amd/csrc/attn.hpp"

struct Launch {
  int64_t kind, grid, waves, u, kg;  // kind 0: none, 1: few rows, 2: many, 3: many in fp32
  int64_t splits, chunk, direct, part_end, ml_end, halves_end, arrived;  // bytes of the workspace up to the end of each
};
static Launch g_launch;
static char* g_base;
static bool g_no_memory, g_error;

static hipError_t fake_malloc(void** p, size_t) {
  if (g_no_memory) {
    g_error = true;  // as the runtime keeps it until it is asked for
    return hipErrorOutOfMemory;
  }
  g_base = reinterpret_cast<char*>((uintptr_t)1 << 40);
  *p = g_base;
  return hipSuccess;
}
static hipError_t fake_free(void*) { return hipSuccess; }
static hipError_t fake_memset(void*, int, size_t) { return hipSuccess; }
static hipError_t fake_wait(hipStream_t) { return hipSuccess; }
static hipError_t fake_last_error() {
  const hipError_t e = g_error ? hipErrorOutOfMemory : hipSuccess;
  g_error = false;
  return e;
}
#define hipMalloc(p, n) fake_malloc(reinterpret_cast<void**>(p), n)
#define hipFree fake_free
#define hipMemset fake_memset
#define hipStreamSynchronize fake_wait
#define hipGetLastError fake_last_error
#include "../activation_residual_compression_amd/csrc/attn_plan.cpp"

static int64_t at(const void* p) { return p ? reinterpret_cast<const char*>(p) - g_base : 0; }
static hipError_t note(int64_t kind, const rc::AttnArgs& a, int64_t grid, int waves, int u, int kg) {
  g_launch = {kind, grid, waves, u, kg, a.splits, a.chunk, a.direct, 0, 0, 0, at(a.arrived)};
  const int64_t rows = kind == 1 ? (int64_t)a.splits * a.kv_heads * a.q_tokens * a.group : grid * 128 * u;
  if (a.splits > 1) {
    g_launch.part_end = at(a.part) + rows * a.dim * 4;
    g_launch.ml_end = at(a.part_ml) + rows * 8;
    if (kind > 1) g_launch.ml_end = at(a.joins) + grid / a.splits * 16;
  }
  if (kind == 3) g_launch.halves_end = at(a.powers) + (int64_t)a.kv_heads * a.kv_tokens * 8;
  return hipSuccess;
}
namespace rc {
hipError_t launch_attn_few(const AttnArgs& a, bool, int waves, int64_t pieces, hipStream_t) { return note(1, a, pieces, waves, 0, 0); }
hipError_t launch_attn_many(const AttnArgs& a, int u, int kg, int64_t grid, hipStream_t) { return note(2, a, grid, 4 * kg, u, kg); }
hipError_t launch_attn_many_f32(const AttnArgs& a, int64_t grid, hipStream_t) { return note(3, a, grid, 4, 1, 1); }
hipError_t launch_attn_join(const AttnJoinArgs&, bool, bool, hipStream_t) {
  g_launch.kind = 4;
  return hipSuccess;
}
}  // namespace rc

extern "C" {
const Launch* choice() { return &g_launch; }
void set_memory(int there) { g_no_memory = !there; }
int last_error() { return (int)fake_last_error(); }
}
