// Decode attention over the paged 4-bit cache, with capped, biased and
// windowed scores, per-key probabilities and the H2O cumulative score (sm_103a).
//
// The mathematics.  A cached key is k = s n + z per group of 32 values (codes
// n in 0..15, kv4.cuh), so with the group's part of q
//   q . k = sum over groups of  s (q . n) + z (sum of q)
// and only q . n is a matrix product: the codes go to the tensor cores as they
// are, the scale and the minimum meet the fp32 result, and no key is ever
// dequantised.  For the values, out = sum_t p_t (s_t n_t + z_t): p_t s_t takes
// the place of p_t in the product with the codes, and sum_t p_t z_t is one
// number per group and head.
//   A nibble is an fp16 number without any conversion: masked into the low
// bits of a 16-bit half it is the subnormal n 2^-24 (or n 2^-20 four bits
// higher), exact in the tensor cores.  Two masks give four such halves of a
// 32-bit word, one shift the other four: 5 operations for 8 values.  The
// powers of two go into q (or into the output).
//   q is scaled per head by a power of two so that its largest magnitude is in
// [2^14, 2^15): bf16 has 8 bits of mantissa, so fp16 then holds it exactly but
// for values 2^-38 of the largest.  p s is scaled per group by a power of two
// taken from the largest s seen so far (p s < 2^14, with p up to 2^8) and
// rounded to fp16: 2^-11 of its value at most, the step's only rounding to 16
// bits; the running maximum, the sums, the scores and the
// output accumulate in fp32.
//
// main kernel: one wave of warps; each takes an equal contiguous share of
//   the tiles of 32 tokens of all (sequence, kv head) pairs, and streams them
//   through a private shared-memory ring with cp.async (no barrier between
//   warps).  Rows are XOR-swizzled in 16-byte chunks, so that ldmatrix (keys)
//   and its transposing form (values: the halves of neighbouring tokens side
//   by side) are free of bank conflicts.  Keys are the left operand (tokens x
//   dims): a thread then holds 4 tokens x 2 heads of a tile and needs the
//   scales of 4 tokens; with q on the left it would be 8 tokens, each read and
//   unpacked by 8 lanes (the first form of this kernel took 119 us instead of
//   88 us at 8 x 32K, 64/8 heads).  p s turns into the second product's layout
//   with movmatrix.  mma.sync, not tcgen05: with at most 16 columns of q the
//   product takes 24 % of the tensor pipe's cycles (8 x 32K), and the
//   codes reach it from registers.
//   A warp whose share ends inside a pair leaves its m, l and partial output.
// finalize kernel: joins the partials of each pair (one CTA per q head), turns
//   the stored scores into probabilities and adds them up over the group's
//   heads (one CTA per 1024 slots).
#include <cuda_fp16.h>

#include "common.cuh"
#include "kv4.cuh"

namespace kvsel {

// Warps of a CTA, one CTA an SM, up to 8 q heads a kv head and above.  Fewer warps with more registers
// (168) beat more of them: at 8 x 32K, 64/8 heads, 12 warps take 73 us, 16 (128 registers, some spilled) 89,
// 20 (96) 134, and 8 with four stages 79.
constexpr int kQdWarps = 12, kQdWarpsWide = 8;
constexpr int kQdTile = 32;                 // tokens of a tile
constexpr int kQdMaxBatch = 1024;
constexpr float kLag = 8.f;                 // see the running maximum
constexpr int kQfSlots = 1024;              // finalize: slots per CTA
constexpr int kQfThreads = 256;

struct __align__(16) QdStage {
  uint8_t k[kQdTile * kQ4CodeBytes];        // chunk c of row r at (c ^ ((r >> 1) & 3))
  uint8_t v[kQdTile * kQ4CodeBytes];
  uint4 ks[kQdTile];                        // {s, z} x 4 of row r
  uint4 vs[kQdTile];
  int32_t pos[kQdTile];
};

struct Decode4Params {
  uint8_t* codes[2];
  uint8_t* scales[2];
  const int32_t* block_table;
  int32_t* seq_lens;
  const __nv_bfloat16* q;
  const __nv_bfloat16* new_kv[2];  // appended rows, or null
  int32_t* pos_map;
  int32_t* next_pos;
  const float* slopes;
  void* out;
  float* logits;        // [B][Hq][max_len] scores in log2 units, or null
  float* probs;         // = logits or null
  float* cum;
  // workspace
  int* status;
  int32_t* eff_len;     // [B] length after the append, -1: rejected
  int32_t* tile_pre;    // [B + 1] tiles of one kv head before sequence b, and of all
  float2* part_ml;      // [warps + pairs][G]
  float* part_o;        // [warps + pairs][G][128]
  float scale, softcap;
  int window, n_sink;
  int B, Hq, Hkv, G, max_len, max_pages, num_pages, page_lg, out_bf16, warps;
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh to about 1e-7 absolute: the series where it converges fast, else from exp.
__device__ __forceinline__ float tanh_acc(float x) {
  const float x2 = x * x;
  const float small = x * fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
  const float e = ex2(2.f * kLog2e * fabsf(x));
  const float big = copysignf(1.f - __fdividef(2.f, e + 1.f), x);
  return fabsf(x) < 0.25f ? small : big;   // e infinite: 2 / inf = 0
}

// D += A (16x16, row) * B (16x8, col), fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16_16816_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                   uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// D = A (16x8, row) * B (8x8, col), tf32 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_tf32_1688_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                   uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 16 bytes into shared memory, zeros if bytes is 0; the cache is read once, so its lines leave L2 first
// (the scores, which the second kernel reads back, stay).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes, uint64_t pol) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes), "l"(pol)
               : "memory");
}

// Tiles of a sequence that hold a key its query may see, in order: the sink
// tiles, then those of the window (all of them without a window, or where
// positions come from a map).
struct TileSet {
  int sink_tiles, win_tile, count;
  __device__ __forceinline__ int slot0(int i) const {
    return (i < sink_tiles ? i : win_tile + (i - sink_tiles)) * kQdTile;
  }
  __device__ __forceinline__ bool holds(int tile) const { return tile < sink_tiles || tile >= win_tile; }
};
__device__ __forceinline__ TileSet tiles_of(int S, int window, int n_sink, bool mapped) {
  const int nt = (S + kQdTile - 1) / kQdTile;
  TileSet t{0, 0, nt};
  if (window > 0 && !mapped && S > window) {
    const int w0 = (S - window) / kQdTile, a = (min(n_sink, S) + kQdTile - 1) / kQdTile;
    if (a < w0) t = TileSet{a, w0, a + nt - w0};
  }
  return t;
}

// Length of sequence b after the append, or -1 if it does not fit.
__device__ __forceinline__ int checked_len(const Decode4Params& P, int b) {
  const int s0 = __ldcg(P.seq_lens + b), add = P.new_kv[0] ? 1 : 0;
  const long long cap = min((long long)P.max_len, (long long)P.max_pages << P.page_lg);
  return s0 < 0 || (long long)s0 + add > cap ? -1 : s0 + add;
}

// kWide: more than 8 q heads a kv head (two blocks of 8 rows).  kMod: scores
// are capped, biased or windowed, or positions come from a map.
template <bool kWide, bool kMod, int kStages>
__global__ void __launch_bounds__((kWide ? kQdWarpsWide : kQdWarps) * 32, 1) kv4_decode_kernel(const Decode4Params P) {
  constexpr int kH = kWide ? 2 : 1, kW = kWide ? kQdWarpsWide : kQdWarps, kThreads = kW * 32;
  extern __shared__ __align__(16) uint8_t qd_smem[];
  __shared__ int s_tiles[kQdMaxBatch + 1];   // exclusive prefix of the sequences' tile counts
  __shared__ int s_len[kQdMaxBatch];
  __shared__ int s_scan[kW];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g8 = lane >> 2, t4 = lane & 3;
  const bool mapped = P.pos_map != nullptr;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the share of this warp
  int carry = 0;
  for (int b0 = 0; b0 < P.B; b0 += kThreads) {
    const int b = b0 + tid;
    int n = 0, S_b = 0;
    if (b < P.B) {
      S_b = checked_len(P, b);
      if (blockIdx.x == 0) {
        P.eff_len[b] = S_b;
        if (S_b < 0) report(P.status, KVSEL_ERR_BAD_INDEX);
      }
      n = S_b > 0 ? tiles_of(S_b, P.window, P.n_sink, mapped).count : 0;
    }
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    int base = carry, sum = carry;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      if (w < warp) base += s_scan[w];
      sum += s_scan[w];
    }
    if (b < P.B) {
      s_tiles[b] = base + x - n;
      s_len[b] = S_b;
      if (blockIdx.x == 0) P.tile_pre[b] = base + x - n;
    }
    carry = sum;
    __syncthreads();
  }
  if (tid == 0) {
    s_tiles[P.B] = carry;
    if (blockIdx.x == 0) P.tile_pre[P.B] = carry;
  }
  __syncthreads();
  const long long T = (long long)carry * P.Hkv;
  const long long N = min((long long)P.warps, T);
  const long long wid = (long long)blockIdx.x * kW + warp;
  if (wid >= N) return;
  long long tile = wid * T / N;
  const long long tile_end = (wid + 1) * T / N;

  QdStage* ring = reinterpret_cast<QdStage*>(qd_smem) + warp * kStages;
  const int page_mask = (1 << P.page_lg) - 1;
  const uint64_t pol = l2_policy_evict_first();
  const uint8_t* codes_k = P.codes[0] + lane * 16;
  const uint8_t* codes_v = P.codes[1] + lane * 16;
  const uint8_t* scales_l = P.scales[lane >> 4] + (lane & 15) * kQ4ScaleBytes;

  // ---- one (sequence, kv head) pair after the other
#pragma unroll 1
  while (tile < tile_end) {
    int b;
    {
      int lo = 0, hi = P.B - 1;   // last b with Hkv * s_tiles[b] <= tile
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((long long)s_tiles[mid] * P.Hkv <= tile) lo = mid;
        else hi = mid - 1;
      }
      b = lo;
    }
    const int nb = s_tiles[b + 1] - s_tiles[b];
    const long long in_b = tile - (long long)s_tiles[b] * P.Hkv;
    const int kvh = int(in_b / nb), i0 = int(in_b - (long long)kvh * nb);
    const int i1 = int(min((long long)nb, i0 + (tile_end - tile)));
    const int S = s_len[b];
    const TileSet ts = tiles_of(S, P.window, P.n_sink, mapped);
    const int32_t* bt = P.block_table + (size_t)b * P.max_pages;
    const size_t rowi = (size_t)b * P.Hkv + kvh;
    int32_t* prow = mapped ? P.pos_map + rowi * P.max_len : nullptr;
    const bool append = P.new_kv[0] != nullptr;
    int pos_q = S - 1;
    float* lg = P.logits ? P.logits + ((size_t)b * P.Hq + kvh * P.G + 2 * t4) * P.max_len + g8 : nullptr;
    if (kMod && mapped) pos_q = append ? __ldcg(P.next_pos + b) : __ldcg(prow + S - 1);

    // q first, so that it is on its way while the copies are set up
    uint4 raw_q[kH][4];
#pragma unroll
    for (int h = 0; h < kH; ++h)
#pragma unroll
      for (int gq = 0; gq < 4; ++gq) {
        raw_q[h][gq] = make_uint4(0, 0, 0, 0);
        if (g8 + 8 * h < P.G)
          raw_q[h][gq] = __ldg(reinterpret_cast<const uint4*>(P.q + ((size_t)b * P.Hq + kvh * P.G + g8 + 8 * h) * kQ4D + 32 * gq + 8 * t4));
      }
    float m[kH][2], l[kH][2], zacc[kH][4][2], o[kH][4][8];
    int e_v[4];               // per group: 2^(e_v - 127) is above every value scale so far
#pragma unroll
    for (int h = 0; h < kH; ++h)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[h][k] = -INFINITY;
        l[h][k] = 0.f;
#pragma unroll
        for (int gq = 0; gq < 4; ++gq) {
          zacc[h][gq][k] = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) o[h][gq][4 * k + i] = 0.f;
        }
      }
#pragma unroll
    for (int gq = 0; gq < 4; ++gq) e_v[gq] = 28;   // scales are 0 or at least 2^-100

    // Page-table entries of a tile's two 16-token halves, read a tile ahead of its copies; copies of
    // tile i into its stage, zeros for bad pages and slots past S.
    auto pages_of = [&](int i, int (&ph)[2]) {
      if (i >= i1) return;
      const int s0 = ts.slot0(i);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int s1 = s0 + 16 * half;
        ph[half] = s1 < S ? __ldg(bt + (s1 >> P.page_lg)) : -1;
      }
    };
    const int c_dst = (lane >> 2) * kQ4CodeBytes + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
    auto fetch = [&](int i, const int (&ph)[2]) {
      QdStage& st = ring[(i - i0) % kStages];
      const int s0 = ts.slot0(i);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const bool ok = unsigned(ph[half]) < unsigned(P.num_pages);
        const uint32_t base = ((uint32_t(ok ? ph[half] : 0) * P.Hkv + kvh) << P.page_lg) + ((s0 + 16 * half) & page_mask);
        const int bytes = ok ? 16 : 0;
        const uint8_t* ck = codes_k + (size_t)base * kQ4CodeBytes;
        const uint8_t* cv = codes_v + (size_t)base * kQ4CodeBytes;
        const uint32_t dk = smem_u32(st.k) + half * 1024 + c_dst, dv = smem_u32(st.v) + half * 1024 + c_dst;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          copy16(dk + k * 512, ck + k * 512, bytes, pol);
          copy16(dv + k * 512, cv + k * 512, bytes, pol);
        }
        const uint8_t* sc = scales_l + (size_t)base * kQ4ScaleBytes;
        copy16(smem_u32((lane >> 4 ? st.vs : st.ks) + 16 * half + (lane & 15)), sc, bytes, pol);
      }
      if (kMod && mapped) {
        const int s = s0 + lane;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(st.pos + lane)), "l"(prow + min(s, S - 1)), "r"(s < S ? 4 : 0) : "memory");
      }
    };
    // ph_in: entries of the tiles already under way, by stage; ph_next: of the next one to fetch
    int ph_in[kStages][2], ph_next[2] = {-1, -1};
#pragma unroll
    for (int k = 0; k < kStages; ++k) ph_in[k][0] = ph_in[k][1] = -1;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) {
      if (i0 + k < i1) {
        pages_of(i0 + k, ph_in[k]);
        fetch(i0 + k, ph_in[k]);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    pages_of(i0 + kStages - 1, ph_next);

    // q: fragments of head g8 (+ 8), scaled by a power of two; group sums and factors of the heads
    // 2 t4, 2 t4 + 1 (+ 8) whose scores this thread holds
    uint32_t qa[kH][4][4];   // per group: {dims 0,4}, {1,5}/16, {2,6}, {3,7}/16 of the thread's word
    uint32_t qz[kH][2];      // sum of q over group t4 of head g8 (+ 8), as two tf32 numbers (22 bits)
    float mult[kH][2], slope[kH][2];
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      const int head = g8 + 8 * h;
      const uint4(&raw)[4] = raw_q[h];
      uint32_t top = 0;
#pragma unroll
      for (int gq = 0; gq < 4; ++gq) {
        const uint32_t r[4] = {raw[gq].x, raw[gq].y, raw[gq].z, raw[gq].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max((r[i] << 16) & 0x7F800000u, r[i] & 0x7F800000u));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // largest magnitude in [2^(e-127), 2^(e-126)), e = top >> 23; q' = q 2^(14-(e-127))
      const int e = max(int(top >> 23), 15);
      const float up = __uint_as_float(uint32_t(268 - e) << 23);   // 13 <= 268 - e <= 253
      float own_sum = 0.f;
#pragma unroll
      for (int gq = 0; gq < 4; ++gq) {
        const uint32_t r[4] = {raw[gq].x, raw[gq].y, raw[gq].z, raw[gq].w};
        float x[8], sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = bf16lo_to_f32(r[i]) * up;
          x[2 * i + 1] = bf16hi_to_f32(r[i]) * up;
          sum += x[2 * i] + x[2 * i + 1];
        }
        qa[h][gq][0] = pack_f16x2(x[0], x[4]);
        qa[h][gq][1] = pack_f16x2(x[1] * 0.0625f, x[5] * 0.0625f);
        qa[h][gq][2] = pack_f16x2(x[2], x[6]);
        qa[h][gq][3] = pack_f16x2(x[3] * 0.0625f, x[7] * 0.0625f);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (gq == t4) own_sum = sum * 0x1p-24f;   // as if it had come out of the product with the codes
      }
      qz[h][0] = __float_as_uint(own_sum) & 0xFFFFE000u;
      qz[h][1] = __float_as_uint(own_sum - __uint_as_float(qz[h][0])) & 0xFFFFE000u;
      // a product with the codes is 2^(141-e-24) times the true one
      float f = P.scale * 0x1p24f * __uint_as_float(uint32_t(e - 14) << 23);
      const float sl = kMod && P.slopes && head < P.G ? __ldg(P.slopes + kvh * P.G + head) * kLog2e : 0.f;
      if (!kMod) f *= kLog2e;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int from = 8 * t4 + 4 * k;   // a lane of head 2 t4 + k
        mult[h][k] = __shfl_sync(0xffffffffu, f, from);
        slope[h][k] = kMod ? __shfl_sync(0xffffffffu, sl, from) : 0.f;
      }
    }

#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();
      const int ph0 = ph_in[0][0], ph1 = ph_in[0][1];
#pragma unroll
      for (int k = 0; k + 1 < kStages; ++k) {
        ph_in[k][0] = ph_in[k + 1][0];
        ph_in[k][1] = ph_in[k + 1][1];
      }
      // the stage read last is free now: the next tile goes there
      if (i + kStages - 1 < i1) {
        fetch(i + kStages - 1, ph_next);
        ph_in[kStages - 2][0] = ph_next[0];
        ph_in[kStages - 2][1] = ph_next[1];
        pages_of(i + kStages, ph_next);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      QdStage& st = ring[(i - i0) % kStages];
      const int s0 = ts.slot0(i);

      // ---- the appended token: quantised here, into the pool and into this tile
      if (append && s0 <= S - 1 && S - 1 < s0 + kQdTile) {
        const int row = S - 1 - s0;
        const int phys = row < 16 ? ph0 : ph1;
        if (unsigned(phys) < unsigned(P.num_pages)) {
          const long long prow_i = ((((long long)phys * P.Hkv + kvh)) << P.page_lg) + ((S - 1) & page_mask);
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const uint2 x = __ldg(reinterpret_cast<const uint2*>(P.new_kv[side] + rowi * kQ4D) + lane);
            const uint32_t raw[2] = {x.x, x.y};
            uint32_t sz;
            const uint32_t codes = q4_group<4>(raw, sz);
            reinterpret_cast<uint16_t*>(P.codes[side] + prow_i * kQ4CodeBytes)[lane] = uint16_t(codes);
            const int off = row * kQ4CodeBytes + (((lane >> 3) ^ ((row >> 1) & 3)) << 4) + (lane & 7) * 2;
            *reinterpret_cast<uint16_t*>((side ? st.v : st.k) + off) = uint16_t(codes);
            if ((lane & 7) == 0) {
              reinterpret_cast<uint32_t*>(P.scales[side] + prow_i * kQ4ScaleBytes)[lane >> 3] = sz;
              reinterpret_cast<uint32_t*>((side ? st.vs : st.ks) + row)[lane >> 3] = sz;
            }
          }
        }
        if (mapped && lane == 0) {
          const int np = __ldcg(P.next_pos + b);
          prow[S - 1] = np;
          st.pos[row] = np;
        }
        __syncwarp();
      }

      // ---- which of the 32 keys are seen (lane t: token t)
      uint32_t vis = 0xffffffffu;
      {
        uint4 own = st.vs[lane];
        const bool inner = s0 + kQdTile <= S && unsigned(ph0) < unsigned(P.num_pages) && unsigned(ph1) < unsigned(P.num_pages);
        if (!inner || (kMod && P.window > 0)) {
          const int s = s0 + lane;
          const bool live = s < S, paged = unsigned(lane < 16 ? ph0 : ph1) < unsigned(P.num_pages);
          bool see = live && paged;
          if (live && !paged) report(P.status, KVSEL_ERR_BAD_INDEX);
          if (kMod && P.window > 0) {
            const int p = mapped ? st.pos[lane] : s;
            see = see && (pos_q - p < P.window || p < P.n_sink);
          }
          vis = __ballot_sync(0xffffffffu, see);
          // what is not seen must not reach the product with p = 0 as NaN or infinity
          if (!see) {
            own = make_uint4(0, 0, 0, 0);
            st.vs[lane] = own;
          }
        }
        // the scales' running exponents
        const uint32_t sc[4] = {own.x & 0x7F80u, own.y & 0x7F80u, own.z & 0x7F80u, own.w & 0x7F80u};
        bool grow = false;
#pragma unroll
        for (int gq = 0; gq < 4; ++gq) grow |= sc[gq] >= uint32_t(e_v[gq]) << 7;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int gq = 0; gq < 4; ++gq) {
            // exponent field + 1: s < 2^(field + 1 - 127); a NaN's field counts as the largest finite one
            const int e = min(int(__reduce_max_sync(0xffffffffu, sc[gq])) >> 7, 253) + 1;
            if (e > e_v[gq]) {
              const float down = __uint_as_float(uint32_t(max(0, 127 - (e - e_v[gq]))) << 23);
#pragma unroll
              for (int h = 0; h < kH; ++h)
#pragma unroll
                for (int k = 0; k < 8; ++k) o[h][gq][k] *= down;
              e_v[gq] = e;
            }
          }
        }
        __syncwarp();
      }
      const uint32_t vis_own = vis >> g8;   // bit 8 r: this thread's token 8 r + g8

      // ---- scores: tokens 8 r + g8 x heads 2 t4, 2 t4 + 1 (+ 8)
      float x[kH][4][2];
      // this lane's row of an 8-row ldmatrix, chunk lane >> 3: rows 8 on have the same swizzle
      const uint32_t ld_off = (lane & 7) * kQ4CodeBytes + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
      const uint32_t k_base = smem_u32(st.k) + ld_off, v_base = smem_u32(st.v) + ld_off;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        // words t4 of groups 0..3 of tokens 16 mt + g8 and + 8
        uint32_t w[2][4];
        uint4 sz[2];
        uint32_t zt[2];   // minimum of group t4 of the two tokens
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          ldsm_x4(k_base + (16 * mt + 8 * r) * kQ4CodeBytes, w[r][0], w[r][1], w[r][2], w[r][3]);
          sz[r] = st.ks[16 * mt + 8 * r + g8];
          zt[r] = reinterpret_cast<const uint32_t*>(st.ks)[(16 * mt + 8 * r) * 4 + lane] & 0xFFFF0000u;
        }
        const uint32_t s0w[4] = {sz[0].x, sz[0].y, sz[0].z, sz[0].w}, s1w[4] = {sz[1].x, sz[1].y, sz[1].z, sz[1].w};
        // the minima's part, z (sum of q): a product over the groups
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          float c[4];
          mma_tf32_1688_zero(c, zt[0], zt[1], zt[0], zt[1], qz[h][0], qz[h][1]);
          x[h][2 * mt][0] = c[0];
          x[h][2 * mt][1] = c[1];
          x[h][2 * mt + 1][0] = c[2];
          x[h][2 * mt + 1][1] = c[3];
        }
#pragma unroll
        for (int gq = 0; gq < 4; ++gq) {
          const uint32_t u0 = w[0][gq] >> 8, u1 = w[1][gq] >> 8;
          const uint32_t a[8] = {w[0][gq] & 0x000F000Fu, w[1][gq] & 0x000F000Fu, w[0][gq] & 0x00F000F0u, w[1][gq] & 0x00F000F0u,
                                 u0 & 0x000F000Fu,       u1 & 0x000F000Fu,       u0 & 0x00F000F0u,       u1 & 0x00F000F0u};
          const float sa = bf16lo_to_f32(s0w[gq]), sb = bf16lo_to_f32(s1w[gq]);
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            float c[4];
            mma_f16_16816_zero(c, a[0], a[1], a[2], a[3], qa[h][gq][0], qa[h][gq][1]);
            mma_f16_16816(c, a[4], a[5], a[6], a[7], qa[h][gq][2], qa[h][gq][3]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              x[h][2 * mt][k] = fmaf(sa, c[k], x[h][2 * mt][k]);
              x[h][2 * mt + 1][k] = fmaf(sb, c[2 + k], x[h][2 * mt + 1][k]);
            }
          }
        }
      }
#pragma unroll
      for (int h = 0; h < kH; ++h) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float y = x[h][r][k] * mult[h][k];
            if (kMod) {
              if (P.softcap > 0.f) y = P.softcap * tanh_acc(__fdividef(y, P.softcap));
              y *= kLog2e;
              if (P.slopes) {
                const int t = 8 * r + g8;
                const int p = mapped ? st.pos[t] : s0 + t;
                y = fmaf(-slope[h][k], fabsf(float(pos_q - p)), y);
              }
            }
            x[h][r][k] = y;
          }
        if (vis != 0xffffffffu) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int k = 0; k < 2; ++k) x[h][r][k] = (vis_own >> (8 * r)) & 1u ? x[h][r][k] : -INFINITY;
        }
        if (P.logits) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (8 * h + 2 * t4 + k < P.G) {
              float* lrow = lg + (size_t)(8 * h + k) * P.max_len + s0;
              if (s0 + kQdTile <= S) {
#pragma unroll
                for (int r = 0; r < 4; ++r) lrow[8 * r] = x[h][r][k];
              } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  if (s0 + 8 * r + g8 < S) lrow[8 * r] = x[h][r][k];
              }
            }
        }
        // m follows the maximum once it lags by more than kLag powers of two: p = 2^(x - m) up to 2^kLag is as
        // good as p up to 1, and most tiles need no reduction over the tokens
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float mx = fmaxf(fmaxf(x[h][0][k], x[h][1][k]), fmaxf(x[h][2][k], x[h][3][k]));
          if (__any_sync(0xffffffffu, mx > m[h][k] + kLag || (m[h][k] == -INFINITY && mx > m[h][k]))) {
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            mx = fmaxf(mx, m[h][k]);
            const float corr = mx == -INFINITY ? 1.f : ex2(m[h][k] - mx);
            m[h][k] = mx;
            l[h][k] *= corr;
#pragma unroll
            for (int gq = 0; gq < 4; ++gq) {
              zacc[h][gq][k] *= corr;
#pragma unroll
              for (int q = 0; q < 4; ++q) o[h][gq][2 * q + k] *= corr;   // columns are heads too
            }
          }
          const float use = m[h][k] == -INFINITY ? 0.f : m[h][k];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[h][r][k] = ex2(x[h][r][k] - use);
            l[h][k] += x[h][r][k];
          }
        }
      }

      // ---- output: (dims x tokens) codes times (tokens x heads) p s, per group
      float inv_e[4];
#pragma unroll
      for (int gq = 0; gq < 4; ++gq) inv_e[gq] = __uint_as_float(uint32_t(260 - e_v[gq]) << 23);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t pb[kH][4][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint4 sz = st.vs[16 * mt + 8 * r + g8];
          const uint32_t sw[4] = {sz.x, sz.y, sz.z, sz.w};
#pragma unroll
          for (int gq = 0; gq < 4; ++gq) {
            const float f = bf16lo_to_f32(sw[gq]) * inv_e[gq], z = bf16hi_to_f32(sw[gq]);
#pragma unroll
            for (int h = 0; h < kH; ++h) {
              const float p0 = x[h][2 * mt + r][0], p1 = x[h][2 * mt + r][1];
              // token g8 x heads 2 t4, + 1 -> tokens 2 t4, + 1 of head g8
              asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(pb[h][gq][r]) : "r"(pack_f16x2(p0 * f, p1 * f)));
              zacc[h][gq][0] = fmaf(p0, z, zacc[h][gq][0]);
              zacc[h][gq][1] = fmaf(p1, z, zacc[h][gq][1]);
            }
          }
        }
        // halves g8 of groups 0..3, tokens 2 t4 and 2 t4 + 1 of the 8 (lo) and the next 8 (hi)
        uint32_t lo[4], hi[4];
        {
          ldsm_x4_t(v_base + 16 * mt * kQ4CodeBytes, lo[0], lo[1], lo[2], lo[3]);
          ldsm_x4_t(v_base + (16 * mt + 8) * kQ4CodeBytes, hi[0], hi[1], hi[2], hi[3]);
        }
#pragma unroll
        for (int gq = 0; gq < 4; ++gq) {
          const uint32_t l8 = lo[gq] >> 8, h8 = hi[gq] >> 8;
          const uint32_t a[8] = {lo[gq] & 0x000F000Fu, lo[gq] & 0x00F000F0u, hi[gq] & 0x000F000Fu, hi[gq] & 0x00F000F0u,
                                 l8 & 0x000F000Fu,     l8 & 0x00F000F0u,     h8 & 0x000F000Fu,     h8 & 0x00F000F0u};
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            float(&o0)[4] = *reinterpret_cast<float(*)[4]>(&o[h][gq][0]);
            float(&o1)[4] = *reinterpret_cast<float(*)[4]>(&o[h][gq][4]);
            mma_f16_16816(o0, a[0], a[1], a[2], a[3], pb[h][gq][0], pb[h][gq][1]);
            mma_f16_16816(o1, a[4], a[5], a[6], a[7], pb[h][gq][0], pb[h][gq][1]);
          }
        }
      }
      __syncwarp();   // this stage may be overwritten
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();

    // ---- the partial result: dims 32 g + 4 g8 + {0..3} of heads 2 t4, 2 t4 + 1
    const long long slot = wid + rowi;   // the staircase of (warp, pair) visits each sum once
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      const int head = 8 * h + 2 * t4;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float lsum = l[h][k];
        lsum += __shfl_xor_sync(0xffffffffu, lsum, 4);
        lsum += __shfl_xor_sync(0xffffffffu, lsum, 8);
        lsum += __shfl_xor_sync(0xffffffffu, lsum, 16);
        if (g8 == 0 && head + k < P.G) P.part_ml[slot * P.G + head + k] = make_float2(m[h][k], lsum);
      }
#pragma unroll
      for (int gq = 0; gq < 4; ++gq) {
        float z[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          z[k] = zacc[h][gq][k];
          z[k] += __shfl_xor_sync(0xffffffffu, z[k], 4);
          z[k] += __shfl_xor_sync(0xffffffffu, z[k], 8);
          z[k] += __shfl_xor_sync(0xffffffffu, z[k], 16);
        }
        // codes were n 2^-24 (dims 0, 2) and n 2^-20 (dims 1, 3), p s was p s 2^(133 - e): undone in
        // two factors so that neither overflows
        const float back = __uint_as_float(uint32_t(e_v[gq] - 6) << 23);
        const float* a = o[h][gq];
        const float c24 = 0x1p24f, c20 = 0x1p20f;
        float* po = P.part_o + (slot * P.G + head) * kQ4D + 32 * gq + 4 * g8;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (head + k < P.G)
            *reinterpret_cast<float4*>(po + k * kQ4D) =
                make_float4(fmaf(a[k] * c24, back, z[k]), fmaf(a[2 + k] * c20, back, z[k]),
                            fmaf(a[4 + k] * c24, back, z[k]), fmaf(a[6 + k] * c20, back, z[k]));
      }
    }
    tile += i1 - i0;
  }
}

// Joins a pair's partials.  blockIdx.x < G: the output of one q head; beyond:
// probabilities and cumulative scores of 1024 slots.
__global__ void __launch_bounds__(kQfThreads) kv4_finalize_kernel(const Decode4Params P) {
  __shared__ float s_m[16], s_inv[16];
  __shared__ float s_red[kQfThreads / 32];
  __shared__ float s_o[kQfThreads / 32][kQ4D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kvh = blockIdx.y, b = blockIdx.z;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool mapped = P.pos_map != nullptr;
  const int S = __ldcg(P.eff_len + b);
  if (S < 0) return;
  const int chunk = int(blockIdx.x) - P.G;
  if (chunk < 0 && blockIdx.x == 0 && kvh == 0 && tid == 0 && P.new_kv[0]) {
    P.seq_lens[b] = S;   // the main kernel is done with the lengths, and this one reads eff_len
    if (P.next_pos) P.next_pos[b] += 1;
  }
  if (chunk >= 0 && chunk * kQfSlots >= S) return;
  if (chunk >= 0 && !P.probs) {   // a chunk that nobody sees adds nothing to the scores
    const TileSet t = tiles_of(S, P.window, P.n_sink, mapped);
    const int first = chunk * (kQfSlots / kQdTile), last = first + kQfSlots / kQdTile - 1;
    if (first >= t.sink_tiles && last < t.win_tile) return;
  }

  const int pre = __ldcg(P.tile_pre + b), tot = __ldcg(P.tile_pre + P.B);
  const TileSet ts = tiles_of(S, P.window, P.n_sink, mapped);
  const long long T = (long long)tot * P.Hkv, N = min((long long)P.warps, T);
  const long long t0 = (long long)pre * P.Hkv + (long long)kvh * ts.count;
  const size_t rowi = (size_t)b * P.Hkv + kvh;
  int w0 = 0, n_part = 0;
  if (ts.count > 0) {   // warp w owns tiles [w T / N, (w + 1) T / N)
    w0 = int(((t0 + 1) * N - 1) / T);
    n_part = int(((t0 + ts.count) * N - 1) / T) - w0 + 1;
  }
  const long long first = (long long)w0 + (long long)rowi;

  if (chunk < 0) {
    const int head = blockIdx.x;
    float mx = -INFINITY;
    for (int i = tid; i < n_part; i += kQfThreads) mx = fmaxf(mx, __ldcg(&P.part_ml[(first + i) * P.G + head]).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) s_red[warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQfThreads / 32; ++w) mx = fmaxf(mx, s_red[w]);
    const float use = mx == -INFINITY ? 0.f : mx;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float lsum = 0.f;
    for (int i = warp; i < n_part; i += kQfThreads / 32) {
      const float2 ml = __ldcg(&P.part_ml[(first + i) * P.G + head]);
      const float f = ex2(ml.x - use);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(P.part_o + ((first + i) * P.G + head) * kQ4D) + lane);
      lsum = fmaf(ml.y, f, lsum);
      acc.x = fmaf(v.x, f, acc.x);
      acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z);
      acc.w = fmaf(v.w, f, acc.w);
    }
    *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = acc;
    __syncthreads();
    if (lane == 0) s_red[warp] = lsum;
    __syncthreads();
    if (tid < kQ4D) {
      float sum = 0.f, v = 0.f;
#pragma unroll
      for (int w = 0; w < kQfThreads / 32; ++w) {
        sum += s_red[w];
        v += s_o[w][tid];
      }
      v = sum == 0.f ? 0.f : v / sum;   // nothing seen: 0
      const size_t at = ((size_t)b * P.Hq + kvh * P.G + head) * kQ4D + tid;
      if (P.out_bf16) static_cast<__nv_bfloat16*>(P.out)[at] = __float2bfloat16(v);
      else static_cast<float*>(P.out)[at] = v;
    }
    return;
  }

  const float* lg = P.logits + ((size_t)b * P.Hq + kvh * P.G) * P.max_len;
  float* crow = P.cum ? P.cum + rowi * P.max_len : nullptr;
  const int new_slot = P.new_kv[0] ? S - 1 : -1;
  constexpr int kPer = kQfSlots / kQfThreads, kFirst = 4;
  const int s0 = chunk * kQfSlots + tid;
  bool use[kPer];
  float sum[kPer], old[kPer], v[kFirst][kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int s = s0 + k * kQfThreads;
    use[k] = s < S && ts.holds(s / kQdTile);
    sum[k] = 0.f;
    old[k] = crow && use[k] && s != new_slot ? __ldcg(crow + s) : 0.f;   // the appended slot starts from 0
  }
  auto load = [&](int h0) {
#pragma unroll
    for (int h = 0; h < kFirst; ++h)
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        v[h][k] = use[k] && h0 + h < P.G ? __ldcs(lg + (size_t)(h0 + h) * P.max_len + s0 + k * kQfThreads) : -INFINITY;
  };
  load(0);   // on their way while the statistics are joined
  // every head's maximum and 1 / sum: 16 threads a head.  Up to 64 partials are read at once; more of them 6 a thread at
  // a time, with a running maximum, as one read after another waits for memory each time.
  {
    const int head = tid >> 4, l16 = tid & 15;
    float mx = -INFINITY, use, sum = 0.f;
    if (n_part <= 64) {
      float2 ml[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = l16 + 16 * k;
        ml[k] = make_float2(-INFINITY, 0.f);
        if (head < P.G && i < n_part) ml[k] = __ldcg(&P.part_ml[(first + i) * P.G + head]);
      }
      mx = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
#pragma unroll
      for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      use = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int k = 0; k < 4; ++k) sum = fmaf(ml[k].y, ex2(ml[k].x - use), sum);
    } else {
      if (head < P.G)
#pragma unroll 1
        for (int i0 = l16; i0 < n_part; i0 += 16 * 6) {
          float2 ml[6];
#pragma unroll
          for (int k = 0; k < 6; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
            if (i0 + 16 * k < n_part) ml[k] = __ldcg(&P.part_ml[(first + i0 + 16 * k) * P.G + head]);
          }
          float top = mx;
#pragma unroll
          for (int k = 0; k < 6; ++k) top = fmaxf(top, ml[k].x);
          const float ref = top == -INFINITY ? 0.f : top;
          sum *= ex2(mx - ref);
#pragma unroll
          for (int k = 0; k < 6; ++k) sum = fmaf(ml[k].y, ex2(ml[k].x - ref), sum);
          mx = top;
        }
      float top = mx;
#pragma unroll
      for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      use = top == -INFINITY ? 0.f : top;
      sum *= ex2(mx - use);
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (l16 == 0) {
      s_m[head] = use;
      s_inv[head] = sum == 0.f ? 0.f : 1.f / sum;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int h0 = 0; h0 < P.G; h0 += kFirst) {
    if (h0 > 0) load(h0);
#pragma unroll
    for (int h = 0; h < kFirst; ++h) {
      if (h0 + h >= P.G) break;
      const float mh = s_m[h0 + h], ih = s_inv[h0 + h];
      float* pr = P.probs ? P.probs + ((size_t)b * P.Hq + kvh * P.G + h0 + h) * P.max_len + s0 : nullptr;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const float p = ex2(v[h][k] - mh) * ih;
        sum[k] += p;
        if (pr && s0 + k * kQfThreads < S) pr[k * kQfThreads] = p;
      }
    }
  }
  if (crow) {
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (use[k]) crow[s0 + k * kQfThreads] = old[k] + sum[k];
  }
}

}  // namespace kvsel

using namespace kvsel;
using namespace kvsel_host;

namespace {

constexpr int kQdStages = 2;

struct Decode4Ws {
  size_t eff_off, pre_off, ml_off, o_off, logits_off, total;
};

// Warps of the main kernel: one CTA an SM.
int decode4_warps(int G) { return sm_count() * (G > 8 ? kQdWarpsWide : kQdWarps); }

// The workspace is sized for the largest grid the device could take; the
// number of SMs is that of the current device.
Decode4Ws decode4_layout(const kvsel_paged_kv4* kv, int batch, int max_len, bool own_logits, int warps) {
  const int G = kv->num_q_heads / kv->num_kv_heads;
  const size_t parts = size_t(warps) + size_t(batch) * kv->num_kv_heads;
  Decode4Ws w;
  w.eff_off = kStatusBytes;
  w.pre_off = align_up(w.eff_off + size_t(batch) * 4, 256);
  w.ml_off = align_up(w.pre_off + size_t(batch + 1) * 4, 256);
  w.o_off = align_up(w.ml_off + parts * G * sizeof(float2), 256);
  w.logits_off = align_up(w.o_off + parts * G * kQ4D * sizeof(float), 256);
  w.total = w.logits_off + (own_logits ? align_up(size_t(batch) * kv->num_q_heads * max_len * sizeof(float), 256) : 0);
  return w;
}

kvsel_status check_shape(const std::string& fn, const kvsel_paged_kv4* kv) {
  if (!kv || kv->num_kv_heads < 1 || kv->num_pages < 1 || kv->num_q_heads < 1 || kv->num_q_heads % kv->num_kv_heads != 0)
    return fail(KVSEL_ERR_INVALID_ARG,
                fn + "a cache descriptor with num_pages, num_kv_heads >= 1 and num_q_heads a multiple of num_kv_heads is required");
  if (page_shift_of(kv->page_size) < 0 || kv->head_dim != kQ4D)
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "only head_dim 128 and page_size 16, 32, 64, 128 or 256 are implemented");
  if (kv->num_q_heads / kv->num_kv_heads > 16)
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "at most 16 q heads per kv head are implemented");
  if ((long long)kv->num_pages * kv->num_kv_heads * kv->page_size >= (1ll << 31))
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "num_pages * num_kv_heads * page_size must be below 2^31");
  return KVSEL_OK;
}

template <bool kWide, bool kMod>
kvsel_status launch_main(const Decode4Params& P, cudaStream_t st) {
  auto* fn = &kv4_decode_kernel<kWide, kMod, kQdStages>;
  constexpr int kW = kWide ? kQdWarpsWide : kQdWarps;
  const int smem = int(sizeof(QdStage)) * kQdStages * kW;
  if (cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(fn), smem); e != cudaSuccess)
    return cuda_fail(e, "kvsel_kv4_decode_attn (attribute)");
  trace_before("kv4_decode", st);
  fn<<<P.warps / kW, kW * 32, smem, st>>>(P);
  cudaError_t e = cudaGetLastError();
  trace_after(st);
  if (e != cudaSuccess) return cuda_fail(e, "kvsel_kv4_decode_attn (launch)");
  return KVSEL_OK;
}

}  // namespace

extern "C" size_t kvsel_kv4_decode_attn_workspace(const kvsel_paged_kv4* kv, int batch, int max_len, int with_probs,
                                                  int with_cum) {
  if (batch < 1 || batch > kQdMaxBatch || max_len < 1 || check_shape("", kv) != KVSEL_OK) return 0;
  return decode4_layout(kv, batch, max_len, with_cum && !with_probs, decode4_warps(kv->num_q_heads / kv->num_kv_heads)).total;
}

extern "C" kvsel_status kvsel_kv4_decode_attn(const kvsel_paged_kv4* kv, const int32_t* block_table, int max_pages,
                                              int32_t* seq_lens, int batch, const void* q, const void* k_new,
                                              const void* v_new, int32_t* pos_map, int32_t* next_pos, float scale,
                                              const kvsel_score_mod* mod, void* out, int out_dtype, float* probs,
                                              float* h2o_cum, int max_len, void* workspace, size_t ws_bytes,
                                              void* stream) {
  const std::string fn = "kvsel_kv4_decode_attn: ";
  if (kvsel_status s = check_shape(fn, kv); s != KVSEL_OK) return s;
  for (const void* p : {kv->k_codes, kv->v_codes, kv->k_scales, kv->v_scales})
    if (!p || !aligned(p, 16)) return fail(KVSEL_ERR_INVALID_ARG, fn + "k_codes, v_codes, k_scales and v_scales (16-byte aligned) are required");
  if (!block_table || !seq_lens || !q || !out || max_pages < 1 || max_len < 1)
    return fail(KVSEL_ERR_INVALID_ARG, fn + "block_table, seq_lens, q, out required; max_pages, max_len >= 1");
  if (batch < 1 || batch > kQdMaxBatch) return fail(KVSEL_ERR_INVALID_ARG, fn + "1 <= batch <= 1024");
  if ((long long)batch * ((max_len + kQdTile - 1ll) / kQdTile) >= (1ll << 31))
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "batch * max_len must be below 2^36");
  if (kv->num_kv_heads > 65535) return fail(KVSEL_ERR_UNSUPPORTED, fn + "at most 65535 kv heads");
  if ((k_new == nullptr) != (v_new == nullptr)) return fail(KVSEL_ERR_INVALID_ARG, fn + "k_new and v_new go together");
  if (pos_map && k_new && !next_pos) return fail(KVSEL_ERR_INVALID_ARG, fn + "pos_map needs next_pos when a token is appended");
  if (out_dtype != KVSEL_BF16 && out_dtype != KVSEL_F32) return fail(KVSEL_ERR_INVALID_ARG, fn + "out_dtype must be KVSEL_BF16 or KVSEL_F32");
  if (!aligned(q, 16) || (k_new && (!aligned(k_new, 16) || !aligned(v_new, 16))))
    return fail(KVSEL_ERR_INVALID_ARG, fn + "q, k_new and v_new must be 16-byte aligned");
  // the comparisons refuse NaN too
  if (mod && (!(mod->softcap >= 0.f) || mod->softcap > 1e30f || mod->window < 0 || mod->n_sink < 0))
    return fail(KVSEL_ERR_INVALID_ARG, fn + "need 0 <= softcap <= 1e30, window >= 0, n_sink >= 0");
  if (!workspace || !aligned(workspace, 256)) return fail(KVSEL_ERR_INVALID_ARG, fn + "a 256-byte aligned workspace is required");
  const int G = kv->num_q_heads / kv->num_kv_heads;
  const int warps = decode4_warps(G);
  const bool own_logits = h2o_cum && !probs;
  const Decode4Ws L = decode4_layout(kv, batch, max_len, own_logits, warps);
  if (ws_bytes < L.total) return fail(KVSEL_ERR_INVALID_ARG, fn + "workspace too small: need " + std::to_string(L.total));

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Decode4Params P;
  P.codes[0] = static_cast<uint8_t*>(kv->k_codes);
  P.codes[1] = static_cast<uint8_t*>(kv->v_codes);
  P.scales[0] = static_cast<uint8_t*>(kv->k_scales);
  P.scales[1] = static_cast<uint8_t*>(kv->v_scales);
  P.block_table = block_table;
  P.seq_lens = seq_lens;
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.new_kv[0] = static_cast<const __nv_bfloat16*>(k_new);
  P.new_kv[1] = static_cast<const __nv_bfloat16*>(v_new);
  P.pos_map = pos_map;
  P.next_pos = k_new ? next_pos : nullptr;
  P.slopes = mod ? mod->slopes : nullptr;
  P.out = out;
  P.logits = probs ? probs : own_logits ? reinterpret_cast<float*>(ws + L.logits_off) : nullptr;
  P.probs = probs;
  P.cum = h2o_cum;
  P.status = reinterpret_cast<int*>(ws);
  P.eff_len = reinterpret_cast<int32_t*>(ws + L.eff_off);
  P.tile_pre = reinterpret_cast<int32_t*>(ws + L.pre_off);
  P.part_ml = reinterpret_cast<float2*>(ws + L.ml_off);
  P.part_o = reinterpret_cast<float*>(ws + L.o_off);
  P.scale = scale;
  P.softcap = mod ? mod->softcap : 0.f;
  P.window = mod ? mod->window : 0;
  P.n_sink = mod ? mod->n_sink : 0;
  P.B = batch;
  P.Hq = kv->num_q_heads;
  P.Hkv = kv->num_kv_heads;
  P.G = G;
  P.max_len = max_len;
  P.max_pages = max_pages;
  P.num_pages = kv->num_pages;
  P.page_lg = 4 + page_shift_of(kv->page_size);
  P.out_bf16 = out_dtype == KVSEL_BF16;
  P.warps = warps;
  const bool modded = P.softcap > 0.f || P.slopes || P.window > 0;
  kvsel_status s = G > 8 ? (modded ? launch_main<true, true>(P, st) : launch_main<true, false>(P, st))
                         : (modded ? launch_main<false, true>(P, st) : launch_main<false, false>(P, st));
  if (s != KVSEL_OK) return s;

  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(G) + (P.logits ? unsigned((max_len + kQfSlots - 1) / kQfSlots) : 0u), kv->num_kv_heads, batch);
  cfg.blockDim = dim3(kQfThreads);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  trace_before("kv4_finalize", st);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_finalize_kernel, P);
  trace_after(st);
  if (e != cudaSuccess) return cuda_fail(e, "kvsel_kv4_decode_attn (finalize launch)");
  return KVSEL_OK;
}
