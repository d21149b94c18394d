// Internal definitions of the paged (full) cache: its device layout and the
// launchers that the host side (kvpop_paged_api.cu) calls.
//
// Device layout of one layer, row-major:
//   pages  [n_pages][Hkv][2][page_size][d]  held elements (key rows, then value
//                                           rows, of one page and head)
//   scales [n_pages][Hkv][2][page_size]     fp32, 8-bit caches only
// One (page, head) pair is one contiguous range, so the keys and values of 16
// tokens arrive in shared memory by one tensor copy.
#pragma once
#include "../../include/kvpop.h"
#include "kvpop_internal.cuh"

namespace kvpop {

constexpr int kMaxGroup = 16;      // query heads per KV head that the attention is built for
constexpr int kAttendRanges = 1024;// most CTAs of one attention launch

// What a kernel needs of one layer's pages.
struct PagedLayer {
  uint8_t* pages;
  float* scales;       // null: rows are held in the element type
  int32_t* err;        // the handle's device error word
  int32_t n_pages, page_shift;   // page_size = 1 << page_shift
  int32_t Hkv;
};

// Rows [batch][token][head][d] with the last dimension contiguous; strides in elements.
struct RowsView {
  uint8_t* p;
  int64_t bs, ts, hs;
};

struct RopeArgs {
  const float* q_weight;
  const float* k_weight;
  const double* inv_freq;   // [rot / 2]
  float eps, scale;
  int rot, interleaved;
};

// One pass over the heads of new tokens.  What is done: queries (when q.p is
// set) and keys are normalised and turned when `turn`; keys and values go to
// the pages when `slots` is set, else keys go to ko.
struct HeadsArgs {
  RowsView q, k, v, qo, ko;
  const int32_t* pos;
  const int32_t* slots;
  RopeArgs rope;
  PagedLayer pg;
  int batch, n_tokens, Hq, Hkv;
};

struct GatherArgs {
  PagedLayer pg;
  const int32_t* table;
  const int32_t* lens;
  int64_t table_stride;
  RowsView k, v;
  int batch, width, n_tokens;
};

struct AttendArgs {
  PagedLayer pg;
  const void* q;
  const int32_t* table;
  const int32_t* lens;
  int64_t table_stride;
  void* out;
  float* lse;
  int batch, width, Hq, G;
  float scale, softcap;
  int window;
  int fixed;        // > 0: parts of kMinShare blocks, this many groups of CTAs for each sequence (set by launch_attend)
};

// Programmatic dependent launch: a kernel's blocks may be set up while the
// kernel before it in the stream still runs.  Every kernel launched so waits
// here before its first access to global memory (until that kernel has ended
// and its writes are visible), and lets the next one be set up.
__device__ __forceinline__ void wait_for_prior_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
int launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess ? 0 : -1;
}

enum HeadsMode : int { HEADS_DENSE = 0, HEADS_APPEND = 1, HEADS_STEP = 2 };

// All return 0, -1 (a CUDA call failed) or -2 (shape not built).
int launch_heads(const HeadsArgs& a, int dtype, int d, int mode, int num_sms, cudaStream_t st);
int launch_gather(const GatherArgs& a, int dtype, int d, cudaStream_t st);
int launch_attend(const CUtensorMap& map, const AttendArgs& a, void* scratch, int dtype, int d, int num_sms,
                  cudaStream_t st);
// Scratch of the attention: partials of kAttendRanges ranges and one arrival
// ticket per unit.  Must be zero before the first launch; each launch leaves
// the tickets zero.
size_t attend_scratch_bytes(int G, int d, int units);
// Tensor map over one layer's pages for the attention's copies of 16 keys and values.
int make_attend_map(CUtensorMap* map, void* pages, int dtype, int d, bool e8, int page_size, int64_t page_heads);
// Sets what the attention kernel of a handle needs on the current device.
int prepare_attend(int dtype, int d, bool e8, int G);

}  // namespace kvpop
