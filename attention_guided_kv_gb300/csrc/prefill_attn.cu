// Attention of prompt tokens over the paged bf16 cache, with capped, biased and
// masked scores, on the fifth-generation tensor cores (sm_103a).
//
// The mathematics: for the rows (query, q head) of one kv head,
//   x = softcap tanh(scale q.k / softcap) - slope |pos_q - j|   (log2 units)
//   O = sum_j 2^(x_j - m) v_j,   l = sum_j 2^(x_j - m),   out = O / l
// in one pass over the keys with a running maximum m.  O is rescaled only when
// m has grown by more than 2^8: until then p = 2^(x - m) up to 256 is as good
// as p up to 1 (bf16 rounds relatively, l and O are fp32).  p is rounded to
// bf16 for the second product, 2^-8 of its value at most; l sums it unrounded.
//
// One CTA takes 256 rows (two tiles of 128; the q heads of a kv head side by
// side, so that K and V are read once for all of them) and the key tiles of
// 128 that any of its rows sees, found from the rows' masks: tiles that all
// rows have masked are not read.
//   warp 8  loads K and V tiles with TMA, 128-byte swizzled, two stages each
//   warp 9  issues tcgen05.mma: S = Q K^T (both from shared memory) and
//           O += P V (P from tensor memory, V as it lies: d contiguous)
//   warps 0-3 and 4-7  one tile each, one thread a row: S out of tensor memory,
//           mask, maximum, exponentials, P back into the columns S had
// A row's 128 scores stay in registers: the softmax warps take 216 each
// (setmaxnreg), warps 8-11 give theirs up.
// Tensor memory is full: 2 x 128 columns of S / P and 2 x 128 of O.  While one
// tile's rows are in the exponentials the other tile's products run.
// Few rows (a chunk of a few tokens): the key tiles are split over several
// CTAs, which leave (m, l, O) in the workspace, and a second kernel joins them.
//
// Keys at or past the sequence's length never matter whatever their pages
// hold: their scores are masked and their V rows zeroed in shared memory (0
// times NaN would be NaN).
#include <type_traits>

#include "common.cuh"
#include "umma.cuh"

namespace kvsel {

constexpr int kPfD = 128;
constexpr int kPfKeys = 128;
constexpr int kPfTileRows = 128;
constexpr int kPfStages = 2;
constexpr int kPfThreads = 384;
constexpr int kPfTileBytes = kPfKeys * kPfD * 2;        // 32 KB: two slabs of 64 columns
constexpr int kPfSlab = kPfKeys * 128;                  // 16 KB
constexpr int kPfSmem = 1024 + (2 + 2 * kPfStages) * kPfTileBytes;
constexpr int kPfMaxSplit = 16;
constexpr float kPfLog2e = 1.4426950408889634f;
constexpr float kPfLn2 = 0.6931471805599453f;
constexpr float kPfSlack = 8.f;                         // m may lag the maximum by this many powers of two

struct PrefillParams {
  const int32_t* block_table;
  const int32_t* seq_lens;
  const __nv_bfloat16* q;
  const int32_t* q_off;
  const float* slopes;
  const int32_t* prefix;
  const int32_t* doc_start;
  void* out;
  float* lse;
  int* status;
  float* part_o;    // [splits][total_q * Hq][128]
  float2* part_ml;  // [splits][total_q * Hq]
  float scale, softcap;
  int window, B, Hq, Hkv, G, max_pages, num_pages, page_lg, total_q, out_bf16, splits;
};

__device__ __forceinline__ float pf_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float pf_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One lane of the warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Descriptor of V as the right operand (K = keys x N = dims, N contiguous,
// 128-byte swizzle): 64-dim slabs kPfSlab apart (LBO), 8-key groups 1024 bytes
// apart (SBO).
__device__ __forceinline__ uint64_t umma_desc_v(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= uint64_t((smem_addr >> 4) & 0x3FFFu);
  d |= uint64_t(kPfSlab >> 4) << 16;
  d |= uint64_t(1024u >> 4) << 32;
  d |= uint64_t(1u) << 46;
  d |= uint64_t(2u) << 61;
  return d;
}

// D[tmem] (+)= A[tmem] * B[smem] for one K = 16 step, issued by one thread.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}

// 32 consecutive 32-bit columns of this thread's TMEM lane, written.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 consecutive fp32 columns of this thread's TMEM lane, not waited for.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
// Values of asynchronous loads may be used only after the wait: this ties 32
// of them to it (volatile statements keep their order).
__device__ __forceinline__ void tmem_tie32(float* v) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])::"memory");
}
// All 128 fp32 columns of this thread's row of S.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&v)[128]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_ld32_async(taddr + 32 * c, v + 32 * c);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_tie32(v + 32 * c);
}

// Two fp32 operations an instruction: (x, y) op ...
__device__ __forceinline__ void fma2(float& dx, float& dy, float ax, float ay, float bx, float by, float cx, float cy) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(dx), "=f"(dy)
      : "f"(ax), "f"(ay), "f"(bx), "f"(by), "f"(cx), "f"(cy));
}
__device__ __forceinline__ void mul2(float& dx, float& dy, float ax, float ay, float bx, float by) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(dx), "=f"(dy)
      : "f"(ax), "f"(ay), "f"(bx), "f"(by));
}
__device__ __forceinline__ void add2(float& dx, float& dy, float ax, float ay, float bx, float by) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(dx), "=f"(dy)
      : "f"(ax), "f"(ay), "f"(bx), "f"(by));
}

// Bits lo..hi (inclusive, both clipped to 0..31) of a word.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  const uint32_t from = lo <= 0 ? ~0u : lo > 31 ? 0u : ~0u << lo;
  const uint32_t to = hi >= 31 ? ~0u : hi < 0 ? 0u : ~0u >> (31 - hi);
  return from & to;
}

// Key tiles that some row of a CTA sees: [a0, a1) and [b0, b1), disjoint, a first.
struct KeyTiles {
  int a0, a1, b0, b1;
  __device__ __forceinline__ int count() const { return (a1 - a0) + (b1 - b0); }
  __device__ __forceinline__ int key0(int i) const { return (i < a1 - a0 ? a0 + i : b0 + i - (a1 - a0)) * kPfKeys; }
};

template <bool kCap, bool kBias>
__global__ void __launch_bounds__(kPfThreads, 1)
prefill_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const PrefillParams P) {
  extern __shared__ uint8_t pf_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pf_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + 2 * kPfTileBytes;
  uint8_t* sV = sK + kPfStages * kPfTileBytes;
  __shared__ uint64_t k_full[kPfStages], v_full[kPfStages], k_empty[kPfStages], v_empty[kPfStages];
  __shared__ uint64_t s_full[2], p_full[2], o_full[2], q_full[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_b, s_tile, s_rng[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  // ---- which rows: CTAs in the order (tile, split, kv head), a sequence's last tile first
  const int kvh = blockIdx.x % P.Hkv, rest = blockIdx.x / P.Hkv;
  const int split = rest % P.splits, want = rest / P.splits;
  if (warp == 0) {
    int before = 0, found = -1, tile = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < P.B && (found < 0 || blockIdx.x == 0); b0 += 32) {   // the first CTA reports on all
      const int b = b0 + lane;
      int nt = 0;
      if (b < P.B) {
        const int a = __ldg(P.q_off + b), e = __ldg(P.q_off + b + 1), S = __ldg(P.seq_lens + b);
        const bool ok = a >= 0 && e >= a && e <= P.total_q && S >= 0 && (long long)S <= ((long long)P.max_pages << P.page_lg);
        if (ok) nt = int(((long long)(e - a) * P.G + 2 * kPfTileRows - 1) / (2 * kPfTileRows));
        else if (blockIdx.x == 0) report(P.status, KVSEL_ERR_BAD_INDEX);
      }
      int x = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const bool mine = want >= before + x - nt && want < before + x;
      const uint32_t who = __ballot_sync(0xffffffffu, mine);
      if (who && found < 0) {
        const int src = __ffs(who) - 1;
        found = b0 + src;
        tile = __shfl_sync(0xffffffffu, before + x - 1 - want, src);
      }
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      s_b = found;
      s_tile = tile;
      s_rng[0] = s_rng[2] = INT32_MAX;
      s_rng[1] = s_rng[3] = 0;
    }
  }
  __syncthreads();
  const int b = s_b;
  if (b < 0) return;
  const int off = __ldg(P.q_off + b), n_q = __ldg(P.q_off + b + 1) - off, S = __ldg(P.seq_lens + b);
  const int rows = n_q * P.G, row0 = s_tile * 2 * kPfTileRows;   // n_q * G < 2^31: checked on the host

  // ---- Q into shared memory, 128-byte swizzled, without waiting; rows past the end are zero
  const int tiles = rows - row0 > kPfTileRows ? 2 : 1;
  if (warp < 8 && (warp >> 2) < tiles) {
    const int t = warp >> 2, ch = tid & 15, r0 = (tid & 127) >> 4, first = row0 + t * kPfTileRows + r0;
    const int di = 8 / P.G, dh = 8 - di * P.G;
    int i = first / P.G, h = first - i * P.G;
    const uint32_t to = smem_u32(sQ) + t * kPfTileBytes + (ch >> 3) * kPfSlab + r0 * 128 + (((ch & 7) ^ r0) << 4);
#pragma unroll 4
    for (int k = 0; k < 16; ++k) {
      const bool have = first + 8 * k < rows;
      const __nv_bfloat16* from = P.q + ((size_t)(off + (have ? i : 0)) * P.Hq + kvh * P.G + (have ? h : 0)) * kPfD + ch * 8;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + k * 1024), "l"(from), "r"(have ? 16 : 0) : "memory");
      i += di;
      h += dh;
      if (h >= P.G) {
        h -= P.G;
        ++i;
      }
    }
  }

  // ---- this thread's row: what it sees
  const int row = row0 + tid;
  const bool in = tid < 2 * kPfTileRows && row < rows;
  int qi = 0, head = 0, pos = 0, jlo = INT32_MIN, jhi = INT32_MAX, jdoc = 0, jpre = 0;
  if (in) {
    qi = row / P.G;
    head = kvh * P.G + (row - qi * P.G);
    pos = S - n_q + qi;
    jdoc = P.doc_start ? max(0, __ldg(P.doc_start + off + qi)) : 0;
    jpre = P.prefix ? min(S, __ldg(P.prefix + b)) : 0;
    jhi = min(pos, S - 1);
    jlo = P.window > 0 ? max(jdoc, pos - P.window + 1) : jdoc;
  }
  if (warp < 8) {
    const bool pre = in && jpre > jdoc, win = in && jhi >= jlo;
    const int a_lo = __reduce_min_sync(0xffffffffu, pre ? jdoc : INT32_MAX);
    const int a_hi = __reduce_max_sync(0xffffffffu, pre ? jpre : 0);
    const int b_lo = __reduce_min_sync(0xffffffffu, win ? jlo : INT32_MAX);
    const int b_hi = __reduce_max_sync(0xffffffffu, win ? jhi + 1 : 0);
    if (lane == 0) {
      atomicMin(&s_rng[0], a_lo);
      atomicMax(&s_rng[1], a_hi);
      atomicMin(&s_rng[2], b_lo);
      atomicMax(&s_rng[3], b_hi);
    }
  }
  if (tid == 0) {
    for (int s = 0; s < kPfStages; ++s) {
      mbar_init(smem_u32(&k_full[s]), 1);
      mbar_init(smem_u32(&v_full[s]), 1);
      mbar_init(smem_u32(&k_empty[s]), 1);
      mbar_init(smem_u32(&v_empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&s_full[t]), 1);
      mbar_init(smem_u32(&p_full[t]), kPfTileRows);
      mbar_init(smem_u32(&o_full[t]), 1);
      mbar_init(smem_u32(&q_full[t]), kPfTileRows);
    }
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, s_tmem, 0);
  KeyTiles kt{0, 0, 0, 0};
  {
    if (s_rng[1] > 0) {
      kt.a0 = s_rng[0] / kPfKeys;
      kt.a1 = (s_rng[1] + kPfKeys - 1) / kPfKeys;
    }
    if (s_rng[3] > 0) {
      kt.b0 = s_rng[2] / kPfKeys;
      kt.b1 = (s_rng[3] + kPfKeys - 1) / kPfKeys;
    }
    if (kt.a1 > kt.a0 && kt.b1 > kt.b0) {
      if (kt.a0 <= kt.b1 && kt.b0 <= kt.a1) kt = KeyTiles{min(kt.a0, kt.b0), max(kt.a1, kt.b1), 0, 0};
      else if (kt.b0 < kt.a0) kt = KeyTiles{kt.b0, kt.b1, kt.a0, kt.a1};
    }
  }
  const int all = kt.count();
  const int i0 = int((long long)split * all / P.splits), n = int((long long)(split + 1) * all / P.splits) - i0;

  // registers: 256 x 216 + 128 x 72 = 64512, the 384 x 168 of the launch
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 8) {
    // ---- producer: a lane per page of the tile
    const int32_t* bt = P.block_table + (size_t)b * P.max_pages;
    const int lg = min(P.page_lg, 7), gran = 1 << lg;   // rows of one copy
    auto resolve = [&](int i) -> int {                  // TMA row of this lane's copy, -1: none
      const int s1 = kt.key0(i0 + i) + (lane << lg);
      if (i >= n || (lane << lg) >= kPfKeys || s1 >= S) return -1;
      int phys = __ldg(bt + (s1 >> P.page_lg));
      if (unsigned(phys) >= unsigned(P.num_pages)) {
        report(P.status, KVSEL_ERR_BAD_INDEX);
        phys = 0;
      }
      return ((phys * P.Hkv + kvh) << P.page_lg) + (s1 & ((1 << P.page_lg) - 1));
    };
    uint64_t pol;                                       // other CTAs read the same keys
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
    int y = resolve(0);
    bool dead = false;
#pragma unroll 1
    for (int i = 0; i < n && !dead; ++i) {
      const int y_next = resolve(i + 1);
      const int s = i % kPfStages;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, y >= 0)) * uint32_t(gran) * 256u;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        uint64_t* full = side ? &v_full[s] : &k_full[s];
        uint64_t* empty = side ? &v_empty[s] : &k_empty[s];
        const CUtensorMap* tm = side ? &tm_v : &tm_k;
        if (!dead && i >= kPfStages) dead = !mbar_wait(smem_u32(empty), ((i / kPfStages) + 1) & 1, P.status);
        dead = __any_sync(0xffffffffu, dead);
        if (dead) break;
        const uint32_t bar = smem_u32(full);
        if (lane == 0) mbar_expect_tx(bar, bytes);
        __syncwarp();
        if (y >= 0) {
          const uint32_t dst = smem_u32((side ? sV : sK) + s * kPfTileBytes) + (uint32_t(lane) << lg) * 128u;
          tma_load_2d(dst, tm, 0, y, bar, pol);
          tma_load_2d(dst + kPfSlab, tm, 64, y, bar, pol);
        }
      }
      y = y_next;
    }
    // (a wait that ran out lasted for seconds after the last copy was started: none is in flight then)
  } else if (warp == 9) {
    // ---- MMA issuer
    const uint32_t id_qk = umma_idesc_bf16_f32(128, kPfKeys), id_pv = umma_idesc_bf16_f32(128, kPfD) | (1u << 16);
    bool ok = true;
    auto wait = [&](uint64_t* bar, int parity) {   // the same answer in every lane
      const bool got = __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, P.status));
      tc_fence_after();
      return got;
    };
    // The operands are the same in every lane and one elected lane issues: a lane picked by its
    // index would have the compiler serialise each instruction over the lanes (80 to 100 cycles
    // each instead of the 64 that it computes).
    const uint64_t dq = umma_desc_sw128(smem_u32(sQ)), dk = umma_desc_sw128(smem_u32(sK)), dv = umma_desc_v(smem_u32(sV));
    auto qk = [&](int t, int i) {
      const uint64_t a = dq + uint64_t(t * (kPfTileBytes >> 4)), k = dk + uint64_t((i % kPfStages) * (kPfTileBytes >> 4));
      const uint32_t d = tbase + t * 128;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t o = uint64_t(((kk >> 2) * kPfSlab + (kk & 3) * 32) >> 4);
          umma_bf16(d, a + o, k + o, id_qk, kk > 0);
        }
        umma_commit(smem_u32(&s_full[t]));
      }
      __syncwarp();
    };
    if (n > 0) {
      ok = wait(&k_full[0], 0);
      for (int t = 0; t < tiles && ok; ++t) {
        ok = wait(&q_full[t], 0);
        if (ok) qk(t, 0);
      }
      if (ok) {
        // a stage is handed back only if another tile comes into it: nothing arrives after the CTA is gone
        if (n > kPfStages && elect_one()) umma_commit(smem_u32(&k_empty[0]));
        __syncwarp();
      }
    }
#pragma unroll 1
    for (int i = 0; i < n && ok; ++i) {
      const int s = i % kPfStages, ph = (i / kPfStages) & 1;
      ok = wait(&v_full[s], ph);
      if (!ok) break;
      const int dead_row = S - kt.key0(i0 + i);          // V rows from here on are not keys
      if (dead_row < kPfKeys) {
        for (int u = dead_row * 8 + lane; u < kPfKeys * 8; u += 32) {
          *reinterpret_cast<uint4*>(sV + s * kPfTileBytes + u * 16) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(sV + s * kPfTileBytes + kPfSlab + u * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
#pragma unroll 1
      for (int t = 0; t < tiles && ok; ++t) {
        ok = wait(&p_full[t], i & 1);
        if (!ok) break;
        const uint64_t v = dv + uint64_t(s * (kPfTileBytes >> 4));
        const uint32_t po = tbase + t * 128, d = po + 256;
        const bool first = i == 0, last = i + 1 == n;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) umma_bf16_ts(d, po + kk * 8, v + uint64_t(kk * (2048 >> 4)), id_pv, !first || kk > 0);
          if (last) umma_commit(smem_u32(&o_full[t]));
        }
        __syncwarp();
        if (i + 1 < n) {
          if (t == 0) {
            ok = wait(&k_full[(i + 1) % kPfStages], ((i + 1) / kPfStages) & 1);
            if (!ok) break;
          }
          qk(t, i + 1);
        }
      }
      if (ok && i + kPfStages < n && elect_one()) umma_commit(smem_u32(&v_empty[s]));
      if (ok && i + 1 + kPfStages < n && elect_one()) umma_commit(smem_u32(&k_empty[(i + 1) % kPfStages]));
      __syncwarp();
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ---- softmax: one thread a row
    const int t = warp >> 2;
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (t < tiles && n > 0) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // Q stores -> tensor-core reads
      mbar_arrive(smem_u32(&q_full[t]));
    }
    const uint32_t lane_addr = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_addr = tbase + lane_addr + t * 128, o_addr = tbase + lane_addr + 256 + t * 128;
    float m = -INFINITY, l = 0.f;
    const float sc = P.scale * kPfLog2e, cap2 = P.softcap * kPfLog2e;
    const float cap_in = kCap ? P.scale / P.softcap : 0.f;
    // softcap log2(e) tanh(cap_in x) ~ x (pc0 + pc1 x^2 + pc2 x^4 + pc3 x^6)
    const float ci2 = cap_in * cap_in, pc0 = 0.999997675f * cap2 * cap_in, pc1 = -0.333206564f * cap2 * cap_in * ci2;
    const float pc2 = 0.131451458f * cap2 * cap_in * ci2 * ci2, pc3 = -0.043372482f * cap2 * cap_in * ci2 * ci2 * ci2;
    const float slope2 = kBias && in ? __ldg(P.slopes + head) * kPfLog2e : 0.f;
    bool ok = true;
    if (t < tiles) {
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        ok = mbar_wait(smem_u32(&s_full[t]), i & 1, P.status);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float x[kPfKeys];
        tmem_ld128(s_addr, x);
        const int t0 = kt.key0(i0 + i);
        const int clo = jlo < t0 ? 0 : jlo - t0, chi = jhi < t0 ? -1 : jhi - t0;      // seen: clo..chi
        const int dlo = jdoc < t0 ? 0 : jdoc - t0, dhi = jpre - t0;                   // and dlo..dhi - 1
        const bool whole = !in || (clo == 0 && chi >= kPfKeys - 1) || (dlo == 0 && dhi >= kPfKeys);
        uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
        const bool part = !__all_sync(0xffffffffu, whole);
        if (part) {
#pragma unroll
          for (int w = 0; w < 4; ++w)
            seen[w] = in ? bit_range(clo - 32 * w, chi - 32 * w) | bit_range(dlo - 32 * w, dhi - 1 - 32 * w) : 0u;
        }
        // softcap tanh(u), u = scale q.k / softcap.  Scores far below the cap (|u| < 0.5, the usual case): an odd
        // polynomial fitted to it there, 1.3e-7 off at most, on the FMA pipe, which has time, where the
        // exponential and the reciprocal would triple the load of the special-function unit.
        bool poly = false;
        if (kCap) {
          float top = fmaxf(fabsf(x[0]), fabsf(x[1]));
#pragma unroll
          for (int c = 2; c < kPfKeys; c += 2) top = max3(top, fabsf(x[c]), fabsf(x[c + 1]));
          poly = __all_sync(0xffffffffu, top * cap_in < 0.5f);
          if (!poly) {
            const float k = 2.f * kPfLog2e * cap_in;
#pragma unroll
            for (int c = 0; c < kPfKeys; ++c) x[c] = fmaf(-2.f * cap2, pf_rcp(pf_ex2(x[c] * k) + 1.f), cap2);
          } else if (kBias) {
#pragma unroll
            for (int c = 0; c < kPfKeys; c += 2) {
              float z0, z1, y0, y1;
              mul2(z0, z1, x[c], x[c + 1], x[c], x[c + 1]);
              fma2(y0, y1, z0, z1, pc3, pc3, pc2, pc2);
              fma2(y0, y1, y0, y1, z0, z1, pc1, pc1);
              fma2(y0, y1, y0, y1, z0, z1, pc0, pc0);
              mul2(x[c], x[c + 1], x[c], x[c + 1], y0, y1);
            }
          }
        }
        if (kBias) {
          const float d = float(pos - t0), base = -slope2 * d, by = kCap ? 1.f : sc;
          // without a prefix no key past the query is seen, and the distance has one sign
          if (!P.prefix || __all_sync(0xffffffffu, pos - t0 >= kPfKeys - 1)) {
#pragma unroll
            for (int c = 0; c < kPfKeys; ++c) x[c] = fmaf(x[c], by, fmaf(slope2, float(c), base));
          } else {
#pragma unroll
            for (int c = 0; c < kPfKeys; ++c) x[c] = fmaf(x[c], by, -slope2 * fabsf(d - float(c)));
          }
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        // Keys that are not seen score -infinity; scores that the polynomial has yet to see stay finite, they
        // only leave the maximum and get p = 0 below.
        const bool late = kCap && !kBias && poly;
        if (part) {
#pragma unroll
          for (int c = 0; c < kPfKeys; c += 2) {
            const float x0 = (seen[c >> 5] >> (c & 31)) & 1u ? x[c] : -INFINITY;
            const float x1 = (seen[c >> 5] >> (c & 31)) & 2u ? x[c + 1] : -INFINITY;
            mx4[(c >> 1) & 3] = max3(mx4[(c >> 1) & 3], x0, x1);
            if (!kCap || kBias) {
              x[c] = x0;
              x[c + 1] = x1;
            } else if (!late) {
              x[c] = x0;
              x[c + 1] = x1;
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < kPfKeys; c += 2) mx4[(c >> 1) & 3] = max3(mx4[(c >> 1) & 3], x[c], x[c + 1]);
        }
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        if (!kCap && !kBias) mx *= sc;                   // sc > 0
        if (kCap && !kBias && poly && mx != -INFINITY)   // x is still raw, and the polynomial is increasing
          mx *= fmaf(fmaf(fmaf(mx * mx, pc3, pc2), mx * mx, pc1), mx * mx, pc0);
        const bool grow = mx > m + kPfSlack || (m == -INFINITY && mx > m);
        if (__any_sync(0xffffffffu, grow)) {
          const float corr = grow ? pf_ex2(m - mx) : 1.f;
          if (grow) m = mx;
          l *= corr;
          if (i > 0) {                                   // every earlier product into O is done: S follows them
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              float o[32];
              uint32_t u[32];
              tmem_ld32(o_addr + 32 * c, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(o[k] * corr);
              tmem_st32(o_addr + 32 * c, u);
            }
          }
        }
        const float use = m == -INFINITY ? 0.f : m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        // Groups of 8 keys: the next group's arguments are computed between the exponentials of this one, so
        // that the FMA pipe and the special-function unit work side by side.
        constexpr int kGrp = 8;
        auto argue = [&](auto late_p, int c0) {
          if constexpr (decltype(late_p)::value) {
#pragma unroll
            for (int c = c0; c < c0 + kGrp; c += 2) {
              float z0, z1, y0, y1;
              mul2(z0, z1, x[c], x[c + 1], x[c], x[c + 1]);
              fma2(y0, y1, z0, z1, pc3, pc3, pc2, pc2);
              fma2(y0, y1, y0, y1, z0, z1, pc1, pc1);
              fma2(y0, y1, y0, y1, z0, z1, pc0, pc0);
              fma2(x[c], x[c + 1], x[c], x[c + 1], y0, y1, -use, -use);
            }
          } else {
#pragma unroll
            for (int c = c0; c < c0 + kGrp; c += 2) {
              if (kCap || kBias) add2(x[c], x[c + 1], x[c], x[c + 1], -use, -use);
              else fma2(x[c], x[c + 1], x[c], x[c + 1], sc, sc, -use, -use);
            }
          }
        };
        auto raise = [&](auto late_p, auto mask_p) {
          uint32_t u[32];
          argue(late_p, 0);
#pragma unroll
          for (int c0 = 0; c0 < kPfKeys; c0 += kGrp) {
            if (c0 + kGrp < kPfKeys) argue(late_p, c0 + kGrp);
#pragma unroll
            for (int c = c0; c < c0 + kGrp; c += 2) {
              float e0 = pf_ex2(x[c]), e1 = pf_ex2(x[c + 1]);
              if constexpr (decltype(mask_p)::value) {
                e0 = (seen[c >> 5] >> (c & 31)) & 1u ? e0 : 0.f;
                e1 = (seen[c >> 5] >> (c & 31)) & 2u ? e1 : 0.f;
              }
              const int k = (c >> 1) & 1;
              add2(sum[2 * k], sum[2 * k + 1], sum[2 * k], sum[2 * k + 1], e0, e1);
              u[(c >> 1) & 31] = pack_bf16x2(e0, e1);
            }
            if ((c0 + kGrp) % 64 == 0) tmem_st32(s_addr + c0 / 64 * 32, u);
          }
        };
        if constexpr (kCap && !kBias) {
          if (!late) raise(std::false_type{}, std::false_type{});
          else if (part) raise(std::true_type{}, std::true_type{});
          else raise(std::true_type{}, std::false_type{});
        } else {
          raise(std::false_type{}, std::false_type{});
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&p_full[t]));
      }
      if (n > 0 && ok) ok = mbar_wait(smem_u32(&o_full[t]), 0, P.status);
      __syncwarp();
      tc_fence_after();
      // The output goes through this tile's Q rows (every product with them is done), so that 16 lanes store a
      // row's 256 bytes together; stored by the row's own thread, 16 bytes of 32 rows at a time, it took 3 us.
      // All four warps come here, and agree on whether every wait was fine.
      uint32_t all;
      asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.and.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                   : "=r"(all)
                   : "r"(1 + t), "r"(uint32_t(ok))
                   : "memory");
      if (all) {
        const float inv = l == 0.f || P.splits > 1 ? 1.f : 1.f / l;
        const bool wide = P.splits > 1 || !P.out_bf16;   // fp32: two passes of 64 dims
        uint8_t* stage = sQ + t * kPfTileBytes;
        const int r = tid & 127, ch = tid & 15, r0 = r >> 4, first = row0 + t * kPfTileRows + r0;
#pragma unroll 1
        for (int pass = 0; pass < (wide ? 2 : 1); ++pass) {
          if (pass) asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
#pragma unroll 1
          for (int c = 0; c < (wide ? 2 : 4); ++c) {
            float o[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0.f;
            if (n > 0) tmem_ld32(o_addr + 64 * pass + 32 * c, o);
            if (l == 0.f) {              // nothing seen: 0
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = 0.f;
            }
            if (wide) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<float4*>(stage + r * 256 + (((8 * c + k) ^ (r & 15)) << 4)) =
                    make_float4(o[4 * k] * inv, o[4 * k + 1] * inv, o[4 * k + 2] * inv, o[4 * k + 3] * inv);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *reinterpret_cast<uint4*>(stage + r * 256 + (((4 * c + k) ^ (r & 15)) << 4)) =
                    make_uint4(pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv), pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                               pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv), pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
            }
          }
          asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
          uint8_t* base = P.splits > 1 ? reinterpret_cast<uint8_t*>(P.part_o + (size_t)split * P.total_q * P.Hq * kPfD)
                                       : static_cast<uint8_t*>(P.out);
          const int di = 8 / P.G, dh = 8 - di * P.G;
          int i = first / P.G, h = first - i * P.G;
#pragma unroll 4
          for (int k = 0; k < 16; ++k) {
            const int rr = r0 + 8 * k;
            if (first + 8 * k < rows) {
              const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 256 + ((ch ^ (rr & 15)) << 4));
              const size_t row_at = (size_t)(off + i) * P.Hq + kvh * P.G + h;
              *reinterpret_cast<uint4*>(base + row_at * (wide ? 512 : 256) + pass * 256 + ch * 16) = v;
            }
            i += di;
            h += dh;
            if (h >= P.G) {
              h -= P.G;
              ++i;
            }
          }
        }
        const size_t at = (size_t)(off + qi) * P.Hq + head;
        if (in && P.splits > 1) P.part_ml[(size_t)split * P.total_q * P.Hq + at] = make_float2(m, l);
        else if (in && P.lse) P.lse[at] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kPfLn2;
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Joins the splits: one warp per (query, q head).
__global__ void __launch_bounds__(256) prefill_join_kernel(const PrefillParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long at = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long n = (long long)P.total_q * P.Hq;
  if (at >= n) return;
  // rows of no sequence, and of one that was rejected, stay as they are
  const int tq = int(at / P.Hq);
  int lo = 0, hi = P.B - 1;
  if (tq >= __ldg(P.q_off + P.B)) return;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(P.q_off + mid) <= tq) lo = mid;
    else hi = mid - 1;
  }
  const int a = __ldg(P.q_off + lo), e = __ldg(P.q_off + lo + 1), S = __ldg(P.seq_lens + lo);
  if (a < 0 || e > P.total_q || tq < a || tq >= e || S < 0 || (long long)S > ((long long)P.max_pages << P.page_lg)) return;
  float2 ml = make_float2(-INFINITY, 0.f);
  if (lane < P.splits) ml = __ldcg(P.part_ml + (size_t)lane * n + at);
  float mx = ml.x;
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float f = ml.y == 0.f ? 0.f : pf_ex2(ml.x - mx);
  float l = ml.y * f;
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < P.splits; ++s) {
    const float fs = __shfl_sync(0xffffffffu, f, s);
    const float4 v = __ldcg(reinterpret_cast<const float4*>(P.part_o + ((size_t)s * n + at) * kPfD) + lane);
    acc.x = fmaf(v.x, fs, acc.x);
    acc.y = fmaf(v.y, fs, acc.y);
    acc.z = fmaf(v.z, fs, acc.z);
    acc.w = fmaf(v.w, fs, acc.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (P.out_bf16)
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(P.out) + at * kPfD)[lane] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  else
    reinterpret_cast<float4*>(static_cast<float*>(P.out) + at * kPfD)[lane] =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (lane == 0 && P.lse) P.lse[at] = l == 0.f ? -INFINITY : (mx + __log2f(l)) * kPfLn2;
}

}  // namespace kvsel

using namespace kvsel;
using namespace kvsel_host;

namespace {

struct PrefillWs {
  int splits;
  size_t ml_off, o_off, total;
};
// CTAs that the packed queries can need at most, and how many parts their keys
// are cut into at most: enough to give every SM a CTA.
PrefillWs prefill_layout(const kvsel_paged_kv* kv, int batch, int total_q) {
  const int G = kv->num_q_heads / kv->num_kv_heads;
  const long long row_tiles = ((long long)total_q * G + 2 * kPfTileRows - 1) / (2 * kPfTileRows) + batch - 1;
  const long long ctas = row_tiles * kv->num_kv_heads;
  long long splits = sm_count() / (ctas > 0 ? ctas : 1);
  if (splits > kPfMaxSplit) splits = kPfMaxSplit;
  if (splits < 1) splits = 1;
  PrefillWs w;
  w.splits = int(splits);
  const size_t rows = size_t(total_q) * kv->num_q_heads;
  w.ml_off = kStatusBytes;
  w.o_off = w.ml_off + (splits > 1 ? align_up(rows * splits * sizeof(float2), 256) : 0);
  w.total = w.o_off + (splits > 1 ? align_up(rows * splits * kPfD * sizeof(float), 256) : 0);
  return w;
}

kvsel_status check_prefill_kv(const std::string& fn, const kvsel_paged_kv* kv) {
  if (!kv || kv->num_kv_heads < 1 || kv->num_pages < 1 || kv->num_q_heads < 1 || kv->num_q_heads % kv->num_kv_heads != 0)
    return fail(KVSEL_ERR_INVALID_ARG,
                fn + "a kv descriptor with num_pages, num_kv_heads >= 1 and num_q_heads a multiple of num_kv_heads is required");
  if (page_shift_of(kv->page_size) < 0 || kv->head_dim != kPfD)
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "only head_dim 128 and page_size 16, 32, 64, 128 or 256 are implemented");
  if (kv->num_q_heads / kv->num_kv_heads > 16)
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "at most 16 q heads per kv head are implemented");
  if ((long long)kv->num_pages * kv->num_kv_heads * kv->page_size >= (1ll << 31))
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "num_pages * num_kv_heads * page_size must be below 2^31");
  return KVSEL_OK;
}

}  // namespace

extern "C" size_t kvsel_prefill_attn_workspace(const kvsel_paged_kv* kv, int batch, int total_q) {
  if (batch < 1 || total_q < 0 || check_prefill_kv("", kv) != KVSEL_OK) return 0;
  return prefill_layout(kv, batch, total_q).total;
}

extern "C" kvsel_status kvsel_prefill_attn(const kvsel_paged_kv* kv, const int32_t* block_table, int max_pages,
                                           const int32_t* seq_lens, int batch, const void* q, const int32_t* q_off,
                                           int total_q, float scale, float softcap, const float* slopes, int window,
                                           const int32_t* prefix, const int32_t* doc_start, void* out, int out_dtype,
                                           float* lse, void* workspace, size_t ws_bytes, void* stream) {
  const std::string fn = "kvsel_prefill_attn: ";
  if (kvsel_status s = check_prefill_kv(fn, kv); s != KVSEL_OK) return s;
  if (!kv->k_pool || !kv->v_pool || !aligned(kv->k_pool, 16) || !aligned(kv->v_pool, 16))
    return fail(KVSEL_ERR_INVALID_ARG, fn + "the K and V pools (16-byte aligned) are required");
  if (!block_table || !seq_lens || !q_off || batch < 1 || max_pages < 1 || total_q < 0)
    return fail(KVSEL_ERR_INVALID_ARG, fn + "block_table, seq_lens, q_off required; batch, max_pages >= 1, total_q >= 0");
  if (total_q > 0 && (!q || !out || !aligned(q, 16) || !aligned(out, 16)))
    return fail(KVSEL_ERR_INVALID_ARG, fn + "q and out (16-byte aligned) are required");
  if (out_dtype != KVSEL_BF16 && out_dtype != KVSEL_F32)
    return fail(KVSEL_ERR_INVALID_ARG, fn + "out_dtype must be KVSEL_BF16 or KVSEL_F32");
  // the comparisons refuse NaN too
  if (!(scale > 0.f) || scale > 1e30f || !(softcap >= 0.f) || softcap > 1e30f || window < 0)
    return fail(KVSEL_ERR_INVALID_ARG, fn + "need 0 < scale <= 1e30, 0 <= softcap <= 1e30, window >= 0");
  if (softcap > 0.f && !(scale / softcap <= 1e30f)) return fail(KVSEL_ERR_INVALID_ARG, fn + "scale / softcap must be at most 1e30");
  if ((long long)total_q * kv->num_q_heads >= (1ll << 31))
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "total_q * num_q_heads must be below 2^31");
  if (!workspace || !aligned(workspace, 256)) return fail(KVSEL_ERR_INVALID_ARG, fn + "a 256-byte aligned workspace is required");
  const PrefillWs L = prefill_layout(kv, batch, total_q);
  if (ws_bytes < L.total) return fail(KVSEL_ERR_INVALID_ARG, fn + "workspace too small: need " + std::to_string(L.total));
  if (total_q == 0) return KVSEL_OK;

  const int G = kv->num_q_heads / kv->num_kv_heads;
  const uint64_t pool_rows = uint64_t(kv->num_pages) * kv->num_kv_heads * kv->page_size;
  const uint32_t box = uint32_t(kv->page_size < kPfKeys ? kv->page_size : kPfKeys);
  CUtensorMap tm_k, tm_v;
  if (!encode_bf16_2d(&tm_k, kv->k_pool, kPfD, pool_rows, kPfD * 2, 64, box) ||
      !encode_bf16_2d(&tm_v, kv->v_pool, kPfD, pool_rows, kPfD * 2, 64, box))
    return fail(KVSEL_ERR_CUDA, fn + "tensor map encoding failed");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  PrefillParams P;
  P.block_table = block_table;
  P.seq_lens = seq_lens;
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.q_off = q_off;
  P.slopes = slopes;
  P.prefix = prefix;
  P.doc_start = doc_start;
  P.out = out;
  P.lse = lse;
  P.status = reinterpret_cast<int*>(ws);
  P.part_ml = reinterpret_cast<float2*>(ws + L.ml_off);
  P.part_o = reinterpret_cast<float*>(ws + L.o_off);
  P.scale = scale;
  P.softcap = softcap;
  P.window = window;
  P.B = batch;
  P.Hq = kv->num_q_heads;
  P.Hkv = kv->num_kv_heads;
  P.G = G;
  P.max_pages = max_pages;
  P.num_pages = kv->num_pages;
  P.page_lg = 4 + page_shift_of(kv->page_size);
  P.total_q = total_q;
  P.out_bf16 = out_dtype == KVSEL_BF16;
  // at least two key tiles a part, by the most that the table can hold
  const long long key_tiles = ((long long)max_pages * kv->page_size + kPfKeys - 1) / kPfKeys;
  P.splits = int(key_tiles / 2 < L.splits ? (key_tiles / 2 > 1 ? key_tiles / 2 : 1) : L.splits);
  auto* fnp = softcap > 0.f ? (slopes ? &prefill_attn_kernel<true, true> : &prefill_attn_kernel<true, false>)
                            : (slopes ? &prefill_attn_kernel<false, true> : &prefill_attn_kernel<false, false>);
  if (cudaError_t e = smem_limit_once(reinterpret_cast<const void*>(fnp), kPfSmem); e != cudaSuccess)
    return cuda_fail(e, "kvsel_prefill_attn (attribute)");
  const long long row_tiles = ((long long)total_q * G + 2 * kPfTileRows - 1) / (2 * kPfTileRows) + batch - 1;
  const long long ctas = row_tiles * kv->num_kv_heads * P.splits;
  if (ctas >= (1ll << 31)) return fail(KVSEL_ERR_UNSUPPORTED, fn + "too many query tiles");
  trace_before("prefill_attn", st);
  fnp<<<unsigned(ctas), kPfThreads, kPfSmem, st>>>(tm_k, tm_v, P);
  cudaError_t e = cudaGetLastError();
  trace_after(st);
  if (e != cudaSuccess) return cuda_fail(e, "kvsel_prefill_attn (launch)");
  if (P.splits > 1) {
    trace_before("prefill_join", st);
    prefill_join_kernel<<<unsigned(((long long)total_q * kv->num_q_heads + 7) / 8), 256, 0, st>>>(P);
    e = cudaGetLastError();
    trace_after(st);
    if (e != cudaSuccess) return cuda_fail(e, "kvsel_prefill_attn (join launch)");
  }
  return KVSEL_OK;
}
