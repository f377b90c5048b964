// The paged 4-bit KV cache: append (quantise), read back, and H2O eviction
// with in-place compaction (sm_103a).  The number format is in kv4.cuh.
//
// append kernel: 16 neighbouring threads take one row (token, kv head), eight
//   values of K and eight of V each: one 16-byte load a side, the group's
//   minimum and maximum over four lanes by shuffles, one 4-byte store of codes
//   a side and, from one lane in four, one of {scale, minimum}.  Nothing is
//   read twice and every store is part of a full 64-byte row: 512 bytes read
//   and 160 written a row.  Where a row goes is looked up by one thread a row.
// read kernel: the inverse, 160 bytes read and 512 written a row.
// evict: the select of h2o_evict.cu (h2o_select_long.cu for long rows), then
//   the kept rows move through shared memory.  Kept lists ascend, so keep[i] >=
//   i: a row's new slot can only be a source of rows before it, and may be
//   written once those have been read.  Up to 7168 kept rows a (sequence, kv
//   head) a cluster of 8 CTAs does that in lock-step rounds, beyond a persistent
//   grid in chunks of 448 rows, claimed in order; one CTA per (sequence, kv
//   head), as the bf16 cache's compaction has it, leaves most SMs idle.
#include "common.cuh"
#include "h2o_select.cuh"
#include "kv4.cuh"

namespace kvsel {

constexpr int kQaThreads = 256;
constexpr int kQaUnroll = 2;                          // rows a thread has in flight
constexpr int kQaStep = kQaThreads / 16 * kQaUnroll;  // rows a CTA has in flight
constexpr int kQaChunk = 256;                         // most rows a CTA looks up at once, one a thread

struct Kv4Params {
  uint8_t* codes[2];   // K, V
  uint8_t* scales[2];
  const int32_t* block_table;
  int32_t* seq_lens;
  const int32_t* tok_off;
  int* status;
  uint32_t* ticket;    // workspace: CTAs that are done with seq_lens
  int Hkv, max_pages, num_pages, page_lg, batch;
  int total;           // packed tokens
  int chunk;           // (token, kv head) rows a CTA takes at a time: a multiple of kQaStep, at most kQaChunk
};

struct AppendParams : Kv4Params {
  const uint4* k;
  const uint4* v;
  int32_t* pos_map;
  int32_t* next_pos;
  float* cum;
  int max_len;
};

struct ReadParams : Kv4Params {
  const int32_t* start;
  uint4* k;
  uint4* v;
};

// The sequence that owns packed token t: the last b with tok_off[b] <= t.
__device__ __forceinline__ int owner_of(const int32_t* off, int batch, int t) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(off + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Run length of sequence b, or -1 if the offsets are not 0 <= ... <= total.
__device__ __forceinline__ int run_of(const Kv4Params& P, int b) {
  const int a = __ldg(P.tok_off + b), e = __ldg(P.tok_off + b + 1);
  return a >= 0 && e >= a && e <= P.total ? e - a : -1;
}

// Pool row of packed (token, kv head) row r's slot, or -1: a row of no sequence
// (nothing is reported) or one that does not fit.  `first`: the slot of a run's
// first token; `limit`: the slots that it may take.
template <class Place>
__device__ __forceinline__ long long pool_row_of(const Kv4Params& P, uint32_t r, int end, Place place) {
  const int t = int(r / uint32_t(P.Hkv)), g = int(r - uint32_t(t) * P.Hkv);
  if (t >= end) return -1;
  const int b = owner_of(P.tok_off, P.batch, t);
  const int n = run_of(P, b), at = t - __ldg(P.tok_off + b);
  long long slot = -1;
  if (n >= 0 && at >= 0 && at < n) slot = place(b, g, n, at);
  int phys = -1;
  if (slot >= 0) phys = __ldg(P.block_table + (size_t)b * P.max_pages + (slot >> P.page_lg));
  if (unsigned(phys) >= unsigned(P.num_pages)) {
    report(P.status, KVSEL_ERR_BAD_INDEX);
    return -1;
  }
  return (((long long)phys * P.Hkv + g) << P.page_lg) + (slot & ((1 << P.page_lg) - 1));
}

__global__ void __launch_bounds__(kQaThreads) kv4_append_kernel(const AppendParams P) {
  __shared__ long long s_row[2][kQaChunk];
  const int tid = threadIdx.x, l16 = tid & 15;
  const uint32_t rows = uint32_t(P.total) * uint32_t(P.Hkv);   // < 2^31 - 2^20: checked on the host
  const long long capacity = (long long)P.max_pages << P.page_lg;
  const int end = __ldg(P.tok_off + P.batch);
  int turn = 0;
#pragma unroll 1
  for (uint32_t c0 = blockIdx.x * P.chunk; c0 < rows; c0 += gridDim.x * P.chunk, turn ^= 1) {
    uint4 kx[kQaUnroll], vx[kQaUnroll];
    auto load = [&](int step) {
#pragma unroll
      for (int u = 0; u < kQaUnroll; ++u) {
        const uint32_t rc = min(c0 + step + u * (kQaThreads / 16) + (tid >> 4), rows - 1);   // every lane takes part in the shuffles
        kx[u] = __ldcs(P.k + size_t(rc) * 16 + l16);
        vx[u] = __ldcs(P.v + size_t(rc) * 16 + l16);
      }
    };
    load(0);
    if (tid < P.chunk && c0 + tid < rows)
      s_row[turn][tid] = pool_row_of(P, c0 + tid, end, [&](int b, int g, int n, int at) -> long long {
        const int S = __ldcg(P.seq_lens + b);
        if (S < 0 || (long long)S + n > capacity || (P.max_len != 0 && (long long)S + n > P.max_len)) return -1;
        const size_t at_row = ((size_t)b * P.Hkv + g) * P.max_len + S + at;
        if (P.pos_map) P.pos_map[at_row] = __ldcg(P.next_pos + b) + at;
        if (P.cum) P.cum[at_row] = 0.0f;
        return (long long)S + at;
      });
    __syncthreads();   // the other buffer is read by the turn before
#pragma unroll 1
    for (int step = 0; step < P.chunk; step += kQaStep) {
      uint32_t sz[kQaUnroll][2], codes[kQaUnroll][2];
#pragma unroll
      for (int u = 0; u < kQaUnroll; ++u) {
        const uint32_t kr[4] = {kx[u].x, kx[u].y, kx[u].z, kx[u].w}, vr[4] = {vx[u].x, vx[u].y, vx[u].z, vx[u].w};
        codes[u][0] = q4_group<8>(kr, sz[u][0]);
        codes[u][1] = q4_group<8>(vr, sz[u][1]);
      }
      if (step + kQaStep < P.chunk) load(step + kQaStep);
#pragma unroll
      for (int u = 0; u < kQaUnroll; ++u) {
        const int i = step + u * (kQaThreads / 16) + (tid >> 4);
        if (c0 + i >= rows) continue;
        const long long row = s_row[turn][i];
        if (row < 0) continue;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          reinterpret_cast<uint32_t*>(P.codes[side] + row * kQ4CodeBytes)[l16] = codes[u][side];
          if ((l16 & 3) == 0) reinterpret_cast<uint32_t*>(P.scales[side] + row * kQ4ScaleBytes)[l16 >> 2] = sz[u][side];
        }
      }
    }
  }
  // the lengths change once every CTA has read them
  __shared__ bool last;
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    last = atomicAdd(P.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int b = tid; b < P.batch; b += kQaThreads) {
    const int n = run_of(P, b), S = __ldcg(P.seq_lens + b);
    if (n < 0 || S < 0 || (long long)S + n > capacity || (P.max_len != 0 && (long long)S + n > P.max_len)) {
      report(P.status, KVSEL_ERR_BAD_INDEX);
      continue;
    }
    P.seq_lens[b] = S + n;
    if (P.next_pos) P.next_pos[b] = __ldcg(P.next_pos + b) + n;
  }
  if (tid == 0) *P.ticket = 0u;
}

__global__ void __launch_bounds__(kQaThreads) kv4_read_kernel(const ReadParams P) {
  __shared__ long long s_row[2][kQaChunk];
  const int tid = threadIdx.x, l16 = tid & 15;
  const uint32_t rows = uint32_t(P.total) * uint32_t(P.Hkv);
  const long long capacity = (long long)P.max_pages << P.page_lg;
  const int end = __ldg(P.tok_off + P.batch);
  int turn = 0;
#pragma unroll 1
  for (uint32_t c0 = blockIdx.x * P.chunk; c0 < rows; c0 += gridDim.x * P.chunk, turn ^= 1) {
    if (tid < P.chunk && c0 + tid < rows)
      s_row[turn][tid] = pool_row_of(P, c0 + tid, end, [&](int b, int, int, int at) -> long long {
        const int S = __ldg(P.seq_lens + b), first = P.start ? __ldg(P.start + b) : 0;
        const long long slot = (long long)first + at;
        return first < 0 || slot >= S || slot >= capacity ? -1 : slot;
      });
    __syncthreads();   // the other buffer is read by the turn before
    uint32_t codes[kQaUnroll][2], sz[kQaUnroll][2];
    long long row[kQaUnroll];
    auto load = [&](int step) {
#pragma unroll
      for (int u = 0; u < kQaUnroll; ++u) {
        const int i = step + u * (kQaThreads / 16) + (tid >> 4);
        row[u] = c0 + i < rows ? s_row[turn][i] : -1;
        if (row[u] < 0) continue;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          codes[u][side] = __ldcs(reinterpret_cast<const uint32_t*>(P.codes[side] + row[u] * kQ4CodeBytes) + l16);
          sz[u][side] = __ldcs(reinterpret_cast<const uint32_t*>(P.scales[side] + row[u] * kQ4ScaleBytes) + (l16 >> 2));
        }
      }
    };
    load(0);
#pragma unroll 1
    for (int step = 0; step < P.chunk; step += kQaStep) {
      uint4 o[kQaUnroll][2];
      bool have[kQaUnroll];
#pragma unroll
      for (int u = 0; u < kQaUnroll; ++u) {
        have[u] = row[u] >= 0;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          const float s = bf16lo_to_f32(sz[u][side]), z = bf16hi_to_f32(sz[u][side]);
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // the code in the mantissa of 2^23 + n, without a conversion
            const float n = __uint_as_float(0x4B000000u | ((codes[u][side] >> (4 * i)) & 15u)) - 8388608.f;
            x[i] = fmaf(n, s, z);
          }
          o[u][side] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                  pack_bf16x2(x[6], x[7]));
        }
      }
      if (step + kQaStep < P.chunk) load(step + kQaStep);
#pragma unroll
      for (int u = 0; u < kQaUnroll; ++u) {
        if (!have[u]) continue;
        const size_t to = size_t(c0 + step + u * (kQaThreads / 16) + (tid >> 4)) * 16 + l16;
        __stcs(P.k + to, o[u][0]);
        __stcs(P.v + to, o[u][1]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// compaction
// ---------------------------------------------------------------------------
constexpr int kQcRows = 448;     // kept rows of a chunk; two CTAs an SM (four of 224 rows: the same at 64 rows, 1.15 times at one)
constexpr int kQcCtas = 2;
constexpr int kQcThreads = 512;
constexpr int kQcUnits = 10;     // 16-byte units of a row: K codes 4, V codes 4, K and V scales
constexpr uint32_t kQcNone = 0xFFFFFFFFu;
constexpr unsigned kQcSpins = 1u << 22;  // polls of the chunks before, each a short sleep: seconds

struct Compact4Params {
  const int32_t* seq_lens;
  const int32_t* block_table;
  const int32_t* keep_slots;
  const int32_t* first_move;
  uint8_t* codes[2];
  uint8_t* scales[2];
  float* cum;
  int32_t* pos_map;
  int* status;
  // workspace, zero when the kernel starts: chunks claimed, per (sequence, kv head) the chunks that are
  // known to have been read from the first on, and a word per chunk that says it has been read
  uint32_t* ticket;
  uint32_t* prefix;
  uint32_t* read;
  int batch, Hkv, max_len, max_pages, num_pages, budget, page_lg, chunks;
};

struct Compact4Smem {
  uint4 unit[kQcRows][kQcUnits];
  uint32_t src[kQcRows], dst[kQcRows];  // pool rows, kQcNone: a bad table entry
  float cum[kQcRows];
  int32_t pos[kQcRows];
  uint32_t ticket;
};

__global__ void __launch_bounds__(kQcThreads) kv4_compact_kernel(const Compact4Params P) {
  extern __shared__ __align__(16) uint8_t qc_smem[];
  Compact4Smem& sm = *reinterpret_cast<Compact4Smem*>(qc_smem);
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kept lists come from the select
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the truncation waits for this kernel
  const int page_mask = (1 << P.page_lg) - 1;
  const uint32_t pairs = uint32_t(P.batch) * P.Hkv, total = pairs * P.chunks;   // < 2^31: checked on the host
  // thread t moves unit t % 10 of rows t / 10, t / 10 + 51, ... (510 of the 512 threads)
  const int w = tid % kQcUnits, r0 = tid / kQcUnits;
  constexpr int kStep = kQcThreads / kQcUnits;
  uint8_t* const pool = w < 4 ? P.codes[0] + w * 16 : w < 8 ? P.codes[1] + (w - 4) * 16 : w == 8 ? P.scales[0] : P.scales[1];
  const uint32_t bytes = w < 8 ? kQ4CodeBytes : kQ4ScaleBytes;
  const unsigned limit = spin_limit(P.status, kQcSpins);
#pragma unroll 1
  while (true) {
    if (tid == 0) sm.ticket = atomicAdd(P.ticket, 1u);
    __syncthreads();
    const uint32_t ticket = sm.ticket;
    if (ticket >= total) break;
    // all rows' first chunks, then their second ones, ...
    const uint32_t pair = ticket % pairs, k = ticket / pairs;
    const int b = int(pair / P.Hkv), kvh = int(pair - uint32_t(b) * P.Hkv);
    const int S = P.seq_lens[b];
    const int i0 = S > P.budget ? P.first_move[pair] + int(k) * kQcRows : P.budget;
    const bool fits = S <= P.max_len && (long long)S <= ((long long)P.max_pages << P.page_lg);
    if (i0 >= P.budget || !fits) {   // nothing to move
      if (!fits && k == 0 && tid == 0) report(P.status, KVSEL_ERR_BAD_INDEX);
      __syncthreads();
      continue;
    }
    const int cnt = min(kQcRows, P.budget - i0);
    const int32_t* keep = P.keep_slots + size_t(pair) * P.budget + i0;
    const int32_t* bt = P.block_table + size_t(b) * P.max_pages;
    float* crow = P.cum + size_t(pair) * P.max_len;
    int32_t* prow = P.pos_map ? P.pos_map + size_t(pair) * P.max_len : nullptr;
    auto pool_row = [&](int slot) -> uint32_t {
      const int phys = __ldg(bt + (slot >> P.page_lg));
      if (unsigned(phys) >= unsigned(P.num_pages)) {
        report(P.status, KVSEL_ERR_BAD_INDEX);
        return kQcNone;
      }
      return ((uint32_t(phys) * P.Hkv + kvh) << P.page_lg) + (slot & page_mask);   // < 2^31: checked on the host
    };
    for (int i = tid; i < cnt; i += kQcThreads) {
      const int src = keep[i];
      sm.src[i] = pool_row(src);
      sm.dst[i] = pool_row(i0 + i);
      sm.cum[i] = __ldcg(crow + src);
      if (prow) sm.pos[i] = __ldcg(prow + src);
    }
    __syncthreads();
    if (r0 < kStep)
      for (int i = r0; i < cnt; i += kStep) {
        const uint32_t row = sm.src[i];
        if (row == kQcNone) continue;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&sm.unit[i][w])), "l"(pool + (size_t)row * bytes) : "memory");
      }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // This chunk has been read.  Its slots may be written once every chunk before it has been read too: kept lists
    // ascend, so keep[i] >= i and only they can have sources there.  A chunk says so before it waits, and chunks are
    // claimed in order, so whatever is waited for is under way.
    volatile uint32_t* read = P.read + size_t(pair) * P.chunks;
    if (tid == 0) {
      __threadfence();
      read[k] = 1u;
    }
    bool go = k == 0;
#pragma unroll 1
    for (unsigned spin = 0; !go && spin < limit; ++spin) {
      const uint32_t from = *(volatile uint32_t*)(P.prefix + pair);
      bool all = true;
      for (uint32_t j = from + tid; j < k; j += kQcThreads) all &= read[j] != 0u;
      // a wait that ran out elsewhere ends this one too (every thread leaves, or none)
      if (__syncthreads_or(tid == 0 && *(volatile int*)P.status == KVSEL_ERR_TIMEOUT)) break;
      go = __syncthreads_and(all);
      if (!go) __nanosleep(100);
    }
    if (!go) {   // the same in every thread
      if (tid == 0) report(P.status, KVSEL_ERR_TIMEOUT);
      break;
    }
    __threadfence();
    if (tid == 0) atomicMax(P.prefix + pair, k + 1);
    if (r0 < kStep)
      for (int i = r0; i < cnt; i += kStep) {
        const uint32_t row = sm.dst[i];
        if (row == kQcNone || sm.src[i] == kQcNone) continue;
        *reinterpret_cast<uint4*>(pool + (size_t)row * bytes) = sm.unit[i][w];
      }
    for (int i = tid; i < cnt; i += kQcThreads) {
      crow[i0 + i] = sm.cum[i];
      if (prow) prow[i0 + i] = sm.pos[i];
    }
    if (gridDim.x >= total) break;   // a chunk a CTA
    __syncthreads();
  }
}

// The move of at most kQkMost kept rows a (sequence, kv head): a cluster of 8 CTAs each, in rounds of 8 x 112 rows.
// A round's rows come into the cluster's shared memory, the cluster waits for all of them and writes them; the next
// round's rows load meanwhile.  64 rows of 32K to 6.5K kept slots: 46.6 us, against 52.8 for the chunks above; of
// 235K kept slots of one row 430 against 41, of 124K of four rows 241 against 59, as only 8 CTAs work on a row here
// (events around the launch).  Between 7168, what a CTA notes the places of at once, and 124K it is not measured.
constexpr int kQkCluster = 8;
constexpr int kQkRows = 112;     // kept rows a CTA stages per round; four CTAs an SM
constexpr int kQkRounds = 8;
constexpr int kQkThreads = 256;
constexpr int kQkMost = kQkCluster * kQkRows * kQkRounds;

struct ClusterSmem {
  uint4 unit[2][kQkRows][kQcUnits];
  uint32_t src[kQkRounds * kQkRows], dst[kQkRounds * kQkRows];  // pool rows, kQcNone: a bad table entry
  float cum[kQkRounds * kQkRows];
  int32_t pos[kQkRounds * kQkRows];
};

__global__ void __launch_bounds__(kQkThreads) kv4_compact_cluster_kernel(const Compact4Params P) {
  extern __shared__ __align__(16) uint8_t qc_smem[];
  ClusterSmem& sm = *reinterpret_cast<ClusterSmem*>(qc_smem);
  const int rank = blockIdx.x % kQkCluster, kvh = blockIdx.x / kQkCluster, b = blockIdx.y, tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kept lists come from the select
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the truncation waits for this kernel
  const int S = P.seq_lens[b];
  if (S <= P.budget) return;  // the same for the whole cluster, as below
  if (S > P.max_len || (long long)S > ((long long)P.max_pages << P.page_lg)) {
    if (tid == 0) report(P.status, KVSEL_ERR_BAD_INDEX);
    return;
  }
  const size_t rowi = size_t(b) * P.Hkv + kvh;
  const int32_t* keep = P.keep_slots + rowi * P.budget;
  const int32_t* bt = P.block_table + size_t(b) * P.max_pages;
  float* crow = P.cum + rowi * P.max_len;
  int32_t* prow = P.pos_map ? P.pos_map + rowi * P.max_len : nullptr;
  const int page_mask = (1 << P.page_lg) - 1;
  auto pool_row = [&](int slot) -> uint32_t {
    const int phys = __ldg(bt + (slot >> P.page_lg));
    if (unsigned(phys) >= unsigned(P.num_pages)) {
      report(P.status, KVSEL_ERR_BAD_INDEX);
      return kQcNone;
    }
    return ((uint32_t(phys) * P.Hkv + kvh) << P.page_lg) + (slot & page_mask);   // < 2^31: checked on the host
  };
  // This CTA's rows of the round that starts at c0: an even share for every CTA of the cluster.
  auto share_of = [&](int c0, int& i0) {
    const int left = min(kQkCluster * kQkRows, P.budget - c0);
    const int share = (left + kQkCluster - 1) / kQkCluster;
    i0 = c0 + rank * share;
    return max(0, min(share, left - rank * share));
  };
  // thread t moves unit t % 10 of rows t / 10, t / 10 + 25, ... (250 of the 256 threads)
  const int w = tid % kQcUnits, r0 = tid / kQcUnits;
  constexpr int kStep = kQkThreads / kQcUnits;
  uint8_t* const pool = w < 4 ? P.codes[0] + w * 16 : w < 8 ? P.codes[1] + (w - 4) * 16 : w == 8 ? P.scales[0] : P.scales[1];
  const uint32_t bytes = w < 8 ? kQ4CodeBytes : kQ4ScaleBytes;
  constexpr int kRound = kQkCluster * kQkRows;
  const int c0 = P.first_move[rowi];
  if (c0 < P.budget) {
    const int rounds = (P.budget - c0 + kRound - 1) / kRound;   // at most kQkRounds: the host's rule
    // where the rows come from and go to
    for (int x = tid; x < rounds * kQkRows; x += kQkThreads) {
      const int k = x / kQkRows, i = x - k * kQkRows;
      int i0;
      if (i < share_of(c0 + k * kRound, i0)) {
        const int src = keep[i0 + i];
        sm.src[x] = pool_row(src);
        sm.dst[x] = pool_row(i0 + i);
        sm.cum[x] = crow[src];
        if (prow) sm.pos[x] = prow[src];
      }
    }
    __syncthreads();
    auto start = [&](int k) {   // round k's rows come into shared memory
      int i0;
      const int cnt = share_of(c0 + k * kRound, i0);
      if (r0 < kStep)
        for (int i = r0; i < cnt; i += kStep) {
          const uint32_t row = sm.src[k * kQkRows + i];
          if (row == kQcNone) continue;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&sm.unit[k & 1][i][w])), "l"(pool + (size_t)row * bytes) : "memory");
        }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    start(0);
#pragma unroll 1
    for (int k = 0; k < rounds; ++k) {
      // the next round's rows are on their way while this one's are written: they lie behind every
      // slot that this round writes
      if (k + 1 < rounds) {
        start(k + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      // all of the round's sources are in shared memory before any of its slots is written (what a CTA
      // reads it has when it arrives, so the barrier need not order memory)
      asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
      int i0;
      const int cnt = share_of(c0 + k * kRound, i0);
      __syncthreads();   // the other threads' copies
      if (r0 < kStep)
        for (int i = r0; i < cnt; i += kStep) {
          const uint32_t row = sm.dst[k * kQkRows + i];
          if (row == kQcNone || sm.src[k * kQkRows + i] == kQcNone) continue;
          *reinterpret_cast<uint4*>(pool + (size_t)row * bytes) = sm.unit[k & 1][i][w];
        }
      for (int i = tid; i < cnt; i += kQkThreads) {
        crow[i0 + i] = sm.cum[k * kQkRows + i];
        if (prow) prow[i0 + i] = sm.pos[k * kQkRows + i];
      }
      __syncthreads();   // the stage is free for the round after the next
    }
  }
}

}  // namespace kvsel

using namespace kvsel;
using namespace kvsel_host;

namespace {

kvsel_status check_kv4(const std::string& fn, const kvsel_paged_kv4* kv) {
  if (!kv || kv->num_kv_heads < 1 || kv->num_pages < 1)
    return fail(KVSEL_ERR_INVALID_ARG, fn + "a cache descriptor with num_pages, num_kv_heads >= 1 is required");
  if (!kv->k_codes || !kv->v_codes || !kv->k_scales || !kv->v_scales)
    return fail(KVSEL_ERR_INVALID_ARG, fn + "k_codes, v_codes, k_scales and v_scales are required");
  for (const void* p : {kv->k_codes, kv->v_codes, kv->k_scales, kv->v_scales})
    if (!aligned(p, 16)) return fail(KVSEL_ERR_INVALID_ARG, fn + "pools must be 16-byte aligned");
  if (page_shift_of(kv->page_size) < 0 || kv->head_dim != kQ4D)
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "only head_dim 128 and page_size 16, 32, 64, 128 or 256 are implemented");
  if ((long long)kv->num_pages * kv->num_kv_heads * kv->page_size >= (1ll << 31))
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "num_pages * num_kv_heads * page_size must be below 2^31");
  return KVSEL_OK;
}

// Rows a CTA takes at a time: few calls' rows are spread over the SMs, many
// rows are looked up 256 at once.  Up to 8 CTAs an SM; more rows are strided over.
int row_chunk(long long rows) {
  const long long even = rows / ((long long)sm_count() * 4) / kQaStep * kQaStep;
  return int(even < kQaStep ? kQaStep : even > kQaChunk ? kQaChunk : even);
}
int row_grid(long long rows, int chunk) {
  const long long want = (rows + chunk - 1) / chunk, most = (long long)sm_count() * 8;
  return int(want < most ? want : most);
}

void fill(Kv4Params& P, const kvsel_paged_kv4* kv, const int32_t* block_table, int max_pages, int32_t* seq_lens, int batch,
          const int32_t* tok_off, int total, void* workspace) {
  P.codes[0] = static_cast<uint8_t*>(kv->k_codes);
  P.codes[1] = static_cast<uint8_t*>(kv->v_codes);
  P.scales[0] = static_cast<uint8_t*>(kv->k_scales);
  P.scales[1] = static_cast<uint8_t*>(kv->v_scales);
  P.block_table = block_table;
  P.seq_lens = seq_lens;
  P.tok_off = tok_off;
  P.status = static_cast<int*>(workspace);
  P.ticket = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
  P.Hkv = kv->num_kv_heads;
  P.max_pages = max_pages;
  P.num_pages = kv->num_pages;
  P.page_lg = 4 + page_shift_of(kv->page_size);
  P.batch = batch;
  P.total = total;
  P.chunk = row_chunk((long long)total * kv->num_kv_heads);
}

// Whether a selection spreads each row over many CTAs.  Whole evictions to 6553 slots, many CTAs a row / one: 1 row of
// 34K slots 64 / 84 us, of 200K 86 / 163; 2 of 34K 72 / 84; 8 of 34K 104 / 96, of 66K 112 / 106, of 200K 131 / 180; 32 of
// 66K 150 / 142, of 200K 206 / 229; 64 of 200K 344 / 307; 128 of 66K 376 / 297.  (3 rows, and more than 64 rows of more than
// 66K or 64 of more than 200K, are not measured.)
constexpr int kLongRow = 32768, kLongRowMany = 100000;   // candidates; the second for more than kLongFew rows
constexpr int kLongFew = 2, kLongRows = 32;
static bool spread_rows(long long candidates, int rows) {
  return rows <= kLongRows && candidates > (rows <= kLongFew ? kLongRow : kLongRowMany);
}

struct Evict4Ws {
  size_t link_off, keep_off, first_off, long_off, sync_off, sync_bytes, total;
  int chunks;
};
// The status block, then the thresholds and candidate counts of the select
// (no candidate lists: the 4-bit decode step does not collect any), what the
// selection of long rows counts in, the kept
// slots, each row's first slot that moves, and what the chunks of the move
// synchronise on (the ticket, a prefix per row, a word per chunk).
Evict4Ws evict4_layout(int batch, int Hkv, int budget) {
  Evict4Ws w;
  const size_t words = align_up(size_t(batch) * Hkv * 4, 256);
  w.link_off = kStatusBytes;
  w.keep_off = w.link_off + 2 * words;
  w.first_off = align_up(w.keep_off + size_t(batch) * Hkv * budget * 4, 256);
  w.chunks = (budget - 1) / kQcRows + 1;
  w.long_off = w.first_off + words;
  w.sync_off = w.long_off + ((long long)batch * Hkv <= kLongRows ? h2o_long_bytes(batch * Hkv) : 0);
  w.sync_bytes = 256 + words + align_up(size_t(batch) * Hkv * w.chunks * 4, 256);
  w.total = w.sync_off + w.sync_bytes;
  return w;
}

}  // namespace

extern "C" size_t kvsel_kv4_append_workspace(const kvsel_paged_kv4* kv, int batch) {
  if (!kv || batch < 1) return 0;
  return kStatusBytes + 256;
}

extern "C" kvsel_status kvsel_kv4_append(const kvsel_paged_kv4* kv, const int32_t* block_table, int max_pages,
                                         int32_t* seq_lens, int batch, const int32_t* tok_off, int total_tokens,
                                         const void* k, const void* v, int32_t* pos_map, int32_t* next_pos,
                                         float* h2o_cum, int max_len, void* workspace, size_t ws_bytes, void* stream) {
  const std::string fn = "kvsel_kv4_append: ";
  if (kvsel_status s = check_kv4(fn, kv); s != KVSEL_OK) return s;
  if (!block_table || !seq_lens || !tok_off || batch < 1 || max_pages < 1 || total_tokens < 0)
    return fail(KVSEL_ERR_INVALID_ARG, fn + "block_table, seq_lens, tok_off required; batch, max_pages >= 1, total_tokens >= 0");
  if (pos_map && !next_pos) return fail(KVSEL_ERR_INVALID_ARG, fn + "pos_map needs next_pos");
  if ((pos_map || h2o_cum) && max_len < 1)
    return fail(KVSEL_ERR_INVALID_ARG, fn + "pos_map and h2o_cum need max_len >= 1");
  if (total_tokens > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16)))
    return fail(KVSEL_ERR_INVALID_ARG, fn + "k and v (16-byte aligned) are required");
  if (!workspace || !aligned(workspace, 256) || ws_bytes < kvsel_kv4_append_workspace(kv, batch))
    return fail(KVSEL_ERR_INVALID_ARG, fn + "a 256-byte aligned workspace of kvsel_kv4_append_workspace() bytes is required");
  if ((long long)total_tokens * kv->num_kv_heads >= (1ll << 31) - (1 << 20))
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "total_tokens * num_kv_heads must be below 2^31 - 2^20");
  if (total_tokens == 0) return KVSEL_OK;
  AppendParams P;
  fill(P, kv, block_table, max_pages, seq_lens, batch, tok_off, total_tokens, workspace);
  P.k = static_cast<const uint4*>(k);
  P.v = static_cast<const uint4*>(v);
  P.pos_map = pos_map;
  P.next_pos = next_pos;
  P.cum = h2o_cum;
  P.max_len = pos_map || h2o_cum ? max_len : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  trace_before("kv4_append", st);
  kv4_append_kernel<<<row_grid((long long)total_tokens * kv->num_kv_heads, P.chunk), kQaThreads, 0, st>>>(P);
  cudaError_t e = cudaGetLastError();
  trace_after(st);
  if (e != cudaSuccess) return cuda_fail(e, "kvsel_kv4_append (launch)");
  return KVSEL_OK;
}

extern "C" kvsel_status kvsel_kv4_read(const kvsel_paged_kv4* kv, const int32_t* block_table, int max_pages,
                                       const int32_t* seq_lens, int batch, const int32_t* tok_off, int total_tokens,
                                       const int32_t* start, void* k_out, void* v_out, void* workspace, size_t ws_bytes,
                                       void* stream) {
  const std::string fn = "kvsel_kv4_read: ";
  if (kvsel_status s = check_kv4(fn, kv); s != KVSEL_OK) return s;
  if (!block_table || !seq_lens || !tok_off || batch < 1 || max_pages < 1 || total_tokens < 0)
    return fail(KVSEL_ERR_INVALID_ARG, fn + "block_table, seq_lens, tok_off required; batch, max_pages >= 1, total_tokens >= 0");
  if (total_tokens > 0 && (!k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16)))
    return fail(KVSEL_ERR_INVALID_ARG, fn + "k_out and v_out (16-byte aligned) are required");
  if (!workspace || !aligned(workspace, 256) || ws_bytes < kStatusBytes)
    return fail(KVSEL_ERR_INVALID_ARG, fn + "a 256-byte aligned workspace of at least 256 bytes is required");
  if ((long long)total_tokens * kv->num_kv_heads >= (1ll << 31) - (1 << 20))
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "total_tokens * num_kv_heads must be below 2^31 - 2^20");
  if (total_tokens == 0) return KVSEL_OK;
  ReadParams P;
  fill(P, kv, block_table, max_pages, const_cast<int32_t*>(seq_lens), batch, tok_off, total_tokens, workspace);
  P.start = start;
  P.k = static_cast<uint4*>(k_out);
  P.v = static_cast<uint4*>(v_out);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  trace_before("kv4_read", st);
  kv4_read_kernel<<<row_grid((long long)total_tokens * kv->num_kv_heads, P.chunk), kQaThreads, 0, st>>>(P);
  cudaError_t e = cudaGetLastError();
  trace_after(st);
  if (e != cudaSuccess) return cuda_fail(e, "kvsel_kv4_read (launch)");
  return KVSEL_OK;
}

extern "C" size_t kvsel_kv4_evict_workspace(const kvsel_paged_kv4* kv, int batch, int budget) {
  if (!kv || batch < 1 || budget < 1 || kv->num_kv_heads < 1) return 0;
  return evict4_layout(batch, kv->num_kv_heads, budget).total;
}

extern "C" kvsel_status kvsel_kv4_evict(const kvsel_paged_kv4* kv, int32_t* block_table, int max_pages, int32_t* seq_lens,
                                        int batch, float* h2o_cum, int32_t* pos_map, int max_len, int budget, int n_sink,
                                        int window, int compact, int32_t* keep_out, int32_t* freed_pages,
                                        void* workspace, size_t ws_bytes, void* stream) {
  const std::string fn = "kvsel_kv4_evict: ";
  if (kvsel_status s = check_kv4(fn, kv); s != KVSEL_OK) return s;
  if (!block_table || !seq_lens || !h2o_cum || batch < 1 || batch > 65535 || max_pages < 1 || max_len < 1)
    return fail(KVSEL_ERR_INVALID_ARG,
                fn + "block_table, seq_lens, h2o_cum required; 1 <= batch <= 65535; max_pages, max_len >= 1");
  if (budget < 1 || n_sink < 0 || window < 0 || (long long)n_sink + window > budget)
    return fail(KVSEL_ERR_INVALID_ARG, fn + "need budget >= 1, n_sink >= 0, window >= 0, n_sink + window <= budget");
  if ((long long)batch * kv->num_kv_heads * ((budget - 1ll) / kQcRows + 1) >= (1ll << 31) - (1 << 20))
    return fail(KVSEL_ERR_UNSUPPORTED, fn + "batch * num_kv_heads * budget is too large");
  if (!workspace || !aligned(workspace, 256))
    return fail(KVSEL_ERR_INVALID_ARG, fn + "a 256-byte aligned workspace is required");
  const Evict4Ws L = evict4_layout(batch, kv->num_kv_heads, budget);
  if (ws_bytes < L.total) return fail(KVSEL_ERR_INVALID_ARG, fn + "workspace too small: need " + std::to_string(L.total));

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  H2OSelectArgs A;
  A.seq_lens = seq_lens;
  A.cum = h2o_cum;
  A.pos_map = pos_map;
  A.keep_slots = reinterpret_cast<int32_t*>(ws + L.keep_off);
  A.keep_out = keep_out;
  A.first_move = reinterpret_cast<int32_t*>(ws + L.first_off);
  A.link = link_layout(workspace, batch * kv->num_kv_heads);
  A.link.key = nullptr;  // counts stay 0, so no list is read
  A.link.pos = nullptr;
  A.status = reinterpret_cast<int*>(ws);
  A.batch = batch;
  A.num_kv_heads = kv->num_kv_heads;
  A.max_len = max_len;
  A.budget = budget;
  A.n_sink = n_sink;
  A.window = window;
  const bool clusters = budget <= kQkMost;
  if (compact && !clusters) {   // before the select, which the move follows closely
    cudaError_t e = cudaMemsetAsync(ws + L.sync_off, 0, L.sync_bytes, st);
    if (e != cudaSuccess) return cuda_fail(e, "kvsel_kv4_evict (clear)");
  }
  const bool long_rows = spread_rows((long long)max_len - n_sink - window, batch * kv->num_kv_heads);
  const kvsel_status sel = long_rows ? launch_h2o_select_long("kvsel_kv4_evict", A, ws + L.long_off, st)
                                     : launch_h2o_select("kvsel_kv4_evict", A, st);
  if (sel != KVSEL_OK) return sel;
  if (!compact) return KVSEL_OK;

  Compact4Params C;
  C.seq_lens = seq_lens;
  C.block_table = block_table;
  C.keep_slots = A.keep_slots;
  C.first_move = A.first_move;
  C.codes[0] = static_cast<uint8_t*>(kv->k_codes);
  C.codes[1] = static_cast<uint8_t*>(kv->v_codes);
  C.scales[0] = static_cast<uint8_t*>(kv->k_scales);
  C.scales[1] = static_cast<uint8_t*>(kv->v_scales);
  C.cum = h2o_cum;
  C.pos_map = pos_map;
  C.status = A.status;
  C.Hkv = kv->num_kv_heads;
  C.max_len = max_len;
  C.max_pages = max_pages;
  C.num_pages = kv->num_pages;
  C.budget = budget;
  C.page_lg = 4 + page_shift_of(kv->page_size);
  C.batch = batch;
  C.chunks = L.chunks;
  C.ticket = reinterpret_cast<uint32_t*>(ws + L.sync_off);
  C.prefix = reinterpret_cast<uint32_t*>(ws + L.sync_off + 256);
  C.read = C.prefix + align_up(size_t(batch) * kv->num_kv_heads * 4, 256) / 4;
  const void* fnp = clusters ? reinterpret_cast<const void*>(kv4_compact_cluster_kernel) : reinterpret_cast<const void*>(kv4_compact_kernel);
  const size_t smem = clusters ? sizeof(ClusterSmem) : sizeof(Compact4Smem);
  if (cudaError_t e = smem_limit_once(fnp, int(smem)); e != cudaSuccess) return cuda_fail(e, "kvsel_kv4_evict (attribute)");
  const long long total = (long long)batch * kv->num_kv_heads * L.chunks, most = (long long)sm_count() * kQcCtas;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = clusters ? dim3(unsigned(kv->num_kv_heads) * kQkCluster, batch) : dim3(unsigned(total < most ? total : most));
  cfg.blockDim = dim3(clusters ? kQkThreads : kQcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kQkCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = clusters ? 2 : 1;
  trace_before("kv4_compact", st);
  cudaError_t e = clusters ? cudaLaunchKernelEx(&cfg, kv4_compact_cluster_kernel, C) : cudaLaunchKernelEx(&cfg, kv4_compact_kernel, C);
  trace_after(st);
  if (e != cudaSuccess) return cuda_fail(e, "kvsel_kv4_evict (compact launch)");

  H2OTruncateArgs T;
  T.seq_lens = seq_lens;
  T.block_table = block_table;
  T.freed = freed_pages;
  T.batch = batch;
  T.max_pages = max_pages;
  T.budget = budget;
  T.max_len = max_len;
  T.page_shift = page_shift_of(kv->page_size);
  return launch_h2o_truncate("kvsel_kv4_evict", T, st);
}
