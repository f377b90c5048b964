// H2O selection of long rows (sm_103a): the keep lists of h2o_select_kernel
// (h2o_evict.cu), with a row spread over many CTAs.
//
// One CTA per row reads 830K scores at the pace of one SM (1005 us; this: 66, events
// around its five launches); here a
// row's candidate slots [n_sink, S - window) are cut into slices, one CTA each:
//   hist kernel, three passes: counts of the order keys' digits (11, 11 and 10
//     bits, from the top), each pass among the keys that share the digits found
//     so far; a pass finds the digit of the one before from its counts.
//   count kernel: keys above and equal to the k-th key, per slice.
//   emit kernel: a slice's offset from the counts before it, then its kept
//     slots in ascending order (lowest slots first among ties), 32 neighbouring
//     slots a warp step.
// Bound by latency: five launches and one read of the scores from HBM, the
// others from L2.
#include "common.cuh"
#include "h2o_select.cuh"

namespace kvsel {

constexpr int kHlThreads = 256;
constexpr int kHlBins = 2048;

struct LongParams {
  const int32_t* seq_lens;
  const float* cum;
  const int32_t* pos_map;
  int32_t* keep_slots;
  int32_t* keep_out;
  int32_t* first_move;
  uint32_t* hint;
  uint32_t* hist;    // [rows][3][kHlBins], zero at the start
  uint2* counts;     // [rows][slices]: above, equal
  int* status;
  int Hkv, max_len, budget, n_sink, window, slices;
};

struct Slice {
  int S, lo, hi, a, e;   // candidates [lo, hi), this slice's [a, e)
  bool select;           // something is evicted
};
__device__ __forceinline__ Slice slice_of(const LongParams& P, int row) {
  Slice s;
  s.S = P.seq_lens[row / P.Hkv];
  s.select = s.S > P.budget && s.S <= P.max_len;
  s.lo = P.n_sink;
  s.hi = s.S - P.window;
  const int n = s.hi - s.lo, per = (n + P.slices - 1) / P.slices;
  const long long a = s.lo + (long long)blockIdx.x * per;
  s.a = int(min(a, (long long)s.hi));
  s.e = int(min(a + per, (long long)s.hi));
  return s;
}

// Digits found by the first `passes` histograms: the keys' prefix, how many of
// the k are still to be found among the keys with it.
struct Found {
  uint32_t prefix, mask, left;
};
__device__ __forceinline__ int hl_shift(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }

__device__ __forceinline__ Found digits(const uint32_t* hist, int passes, uint32_t k, uint32_t* tmp, uint32_t* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Found f{0u, 0u, k};
  constexpr int kEach = kHlBins / kHlThreads;
#pragma unroll 1
  for (int p = 0; p < passes; ++p) {
    uint32_t c[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {   // bins from the top down
      c[i] = __ldcg(hist + p * kHlBins + (kHlBins - 1 - (tid * kEach + i)));
      sum += c[i];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) tmp[warp] = incl;
    __syncthreads();
    uint32_t before = incl - sum;
#pragma unroll
    for (int w = 0; w < kHlThreads / 32; ++w)
      if (w < warp) before += tmp[w];
    if (before < f.left && f.left <= before + sum) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (before < f.left && f.left <= before + c[i]) {
          out[0] = kHlBins - 1 - (tid * kEach + i);
          out[1] = before;
        }
        before += c[i];
      }
    }
    __syncthreads();
    f.prefix |= out[0] << hl_shift(p);
    f.mask |= (p == 2 ? 0x3FFu : 0x7FFu) << hl_shift(p);
    f.left -= out[1];
    __syncthreads();
  }
  return f;
}

__global__ void __launch_bounds__(kHlThreads) h2o_long_hist_kernel(const LongParams P, int pass) {
  __shared__ uint32_t s_hist[kHlBins];
  __shared__ uint32_t s_tmp[kHlThreads / 32], s_out[2];
  const int row = blockIdx.y, tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Slice sl = slice_of(P, row);
  if (pass == 0 && blockIdx.x == 0 && tid == 0) {
    if (sl.S < 0 || sl.S > P.max_len) report(P.status, KVSEL_ERR_BAD_INDEX);
    P.first_move[row] = sl.S <= P.budget ? sl.S : P.budget;
  }
  const int k = P.budget - P.n_sink - P.window;
  if (!sl.select || k == 0) return;
  for (int i = tid; i < kHlBins; i += kHlThreads) s_hist[i] = 0u;
  uint32_t* hist = P.hist + size_t(row) * 3 * kHlBins;
  const Found f = digits(hist, pass, uint32_t(k), s_tmp, s_out);
  __syncthreads();
  const float* score = P.cum + size_t(row) * P.max_len;
  const int shift = hl_shift(pass);
  const uint32_t digit = pass == 2 ? 0x3FFu : 0x7FFu;
#pragma unroll 8
  for (int i = sl.a + tid; i < sl.e; i += kHlThreads) {
    const uint32_t u = order_key(__ldcg(score + i));
    if ((u & f.mask) == f.prefix) atomicAdd(&s_hist[(u >> shift) & digit], 1u);
  }
  __syncthreads();
  for (int i = tid; i < kHlBins; i += kHlThreads)
    if (const uint32_t c = s_hist[i]) atomicAdd(hist + pass * kHlBins + i, c);
}

// A slice's warps own contiguous runs of whole 32-slot steps.
struct WarpRun {
  int a, e;
};
__device__ __forceinline__ WarpRun run_of_warp(const Slice& sl) {
  const int steps = (sl.e - sl.a + 31) / 32, per = (steps + kHlThreads / 32 - 1) / (kHlThreads / 32);
  const int a = sl.a + (threadIdx.x >> 5) * per * 32;
  return WarpRun{min(a, sl.e), min(a + per * 32, sl.e)};
}

__global__ void __launch_bounds__(kHlThreads) h2o_long_count_kernel(const LongParams P) {
  __shared__ uint32_t s_tmp[kHlThreads / 32], s_out[2], s_gt, s_eq;
  const int row = blockIdx.y, tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Slice sl = slice_of(P, row);
  const int k = P.budget - P.n_sink - P.window;
  if (!sl.select || k == 0) return;
  if (tid == 0) s_gt = s_eq = 0u;
  const uint32_t T = digits(P.hist + size_t(row) * 3 * kHlBins, 3, uint32_t(k), s_tmp, s_out).prefix;
  const float* score = P.cum + size_t(row) * P.max_len;
  uint32_t gt = 0, eq = 0;
#pragma unroll 8
  for (int i = sl.a + tid; i < sl.e; i += kHlThreads) {
    const uint32_t u = order_key(__ldcg(score + i));
    gt += u > T;
    eq += u == T;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if ((tid & 31) == 0) {
    atomicAdd(&s_gt, gt);
    atomicAdd(&s_eq, eq);
  }
  __syncthreads();
  if (tid == 0) P.counts[size_t(row) * P.slices + blockIdx.x] = make_uint2(s_gt, s_eq);
}

__global__ void __launch_bounds__(kHlThreads) h2o_long_emit_kernel(const LongParams P) {
  __shared__ uint32_t s_tmp[kHlThreads / 32], s_out[2], s_gt[kHlThreads / 32], s_eq[kHlThreads / 32], s_before[2];
  const int row = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Slice sl = slice_of(P, row);
  if (sl.S < 0 || sl.S > P.max_len) return;
  const int32_t* prow = P.pos_map ? P.pos_map + size_t(row) * P.max_len : nullptr;
  int32_t* keep = P.keep_slots + size_t(row) * P.budget;
  int32_t* kout = P.keep_out ? P.keep_out + size_t(row) * P.budget : nullptr;
  const int all = blockIdx.x * kHlThreads + tid, stride = P.slices * kHlThreads;
  if (!sl.select) {
    for (int i = all; i < P.budget; i += stride) {
      const int slot = i < sl.S ? i : -1;
      keep[i] = slot;
      if (kout) kout[i] = slot < 0 ? -1 : (prow ? prow[slot] : slot);
    }
    return;
  }
  int first = P.budget;
  auto put = [&](int o, int slot) {
    keep[o] = slot;
    if (kout) kout[o] = prow ? prow[slot] : slot;
    if (slot != o) first = min(first, o);
  };
  for (int i = all; i < P.n_sink; i += stride) put(i, i);
  for (int i = all; i < P.window; i += stride) put(P.budget - P.window + i, sl.S - P.window + i);
  const int k = P.budget - P.n_sink - P.window;
  if (k > 0) {
    if (tid < 2) s_before[tid] = 0u;
    const Found f = digits(P.hist + size_t(row) * 3 * kHlBins, 3, uint32_t(k), s_tmp, s_out);
    const uint32_t T = f.prefix, need_eq = f.left;
    if (blockIdx.x == 0 && tid == 0) P.hint[row] = T;
    // kept slots before this slice
    uint32_t g0 = 0, e0 = 0;
    for (int i = tid; i < int(blockIdx.x); i += kHlThreads) {
      const uint2 c = __ldcg(P.counts + size_t(row) * P.slices + i);
      g0 += c.x;
      e0 += c.y;
    }
    g0 = __reduce_add_sync(0xffffffffu, g0);
    e0 = __reduce_add_sync(0xffffffffu, e0);
    if (lane == 0) {
      atomicAdd(&s_before[0], g0);
      atomicAdd(&s_before[1], e0);
    }
    const float* score = P.cum + size_t(row) * P.max_len;
    const WarpRun run = run_of_warp(sl);
    uint32_t gt = 0, eq = 0;
#pragma unroll 4
    for (int i = run.a + lane; i < run.e; i += 32) {
      const uint32_t u = order_key(__ldcg(score + i));
      gt += u > T;
      eq += u == T;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
      s_gt[warp] = gt;
      s_eq[warp] = eq;
    }
    __syncthreads();
    uint32_t g_seen = s_before[0], e_seen = s_before[1];
    for (int w = 0; w < warp; ++w) {
      g_seen += s_gt[w];
      e_seen += s_eq[w];
    }
    uint32_t lt;
    asm("mov.u32 %0, %%lanemask_lt;" : "=r"(lt));
#pragma unroll 1
    for (int i0 = run.a; i0 < run.e; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t u = i < run.e ? order_key(__ldcg(score + i)) : 0u;
      const bool is_gt = i < run.e && u > T, is_eq = i < run.e && u == T;
      const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
      const uint32_t e_rank = e_seen + __popc(be & lt);
      if (is_gt || (is_eq && e_rank < need_eq)) {
        const uint32_t o = g_seen + __popc(bg & lt) + min(e_rank, need_eq);
        if (o < uint32_t(k)) put(P.n_sink + int(o), i);
      }
      g_seen += __popc(bg);
      e_seen += __popc(be);
    }
  }
  first = __reduce_min_sync(0xffffffffu, first);
  if (lane == 0 && first < P.budget) atomicMin(P.first_move + row, first);
}

}  // namespace kvsel

using namespace kvsel;

namespace kvsel_host {

constexpr int kMostSlices = 128;

size_t h2o_long_bytes(int rows) {
  return align_up(size_t(rows) * 3 * kHlBins * sizeof(uint32_t), 256) + align_up(size_t(rows) * kMostSlices * sizeof(uint2), 256);
}

kvsel_status launch_h2o_select_long(const char* fn, const H2OSelectArgs& a, void* scratch, cudaStream_t st) {
  const int rows = a.batch * a.num_kv_heads;
  const std::string name(fn);
  LongParams P;
  P.seq_lens = a.seq_lens;
  P.cum = a.cum;
  P.pos_map = a.pos_map;
  P.keep_slots = a.keep_slots;
  P.keep_out = a.keep_out;
  P.first_move = a.first_move;
  P.hint = a.link.hint;
  P.hist = static_cast<uint32_t*>(scratch);
  P.counts = reinterpret_cast<uint2*>(static_cast<uint8_t*>(scratch) + align_up(size_t(rows) * 3 * kHlBins * sizeof(uint32_t), 256));
  P.status = a.status;
  P.Hkv = a.num_kv_heads;
  P.max_len = a.max_len;
  P.budget = a.budget;
  P.n_sink = a.n_sink;
  P.window = a.window;
  const int want = 4 * sm_count() / rows;   // four CTAs an SM
  P.slices = want < 1 ? 1 : want > kMostSlices ? kMostSlices : want;
  cudaError_t e = cudaMemsetAsync(P.hist, 0, size_t(rows) * 3 * kHlBins * sizeof(uint32_t), st);
  if (e != cudaSuccess) return cuda_fail(e, (name + " (clear)").c_str());
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.slices, rows);
  cfg.blockDim = dim3(kHlThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  for (int pass = 0; pass < 5; ++pass) {
    trace_before(pass < 3 ? "h2o_long_hist" : pass == 3 ? "h2o_long_count" : "h2o_long_emit", st);
    e = pass < 3    ? cudaLaunchKernelEx(&cfg, h2o_long_hist_kernel, P, pass)
        : pass == 3 ? cudaLaunchKernelEx(&cfg, h2o_long_count_kernel, P)
                    : cudaLaunchKernelEx(&cfg, h2o_long_emit_kernel, P);
    trace_after(st);
    if (e != cudaSuccess) return cuda_fail(e, (name + " (select launch)").c_str());
  }
  return KVSEL_OK;
}

}  // namespace kvsel_host
