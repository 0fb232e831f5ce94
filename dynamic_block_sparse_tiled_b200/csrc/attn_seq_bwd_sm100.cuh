// attn_seq_bwd_sm100.cuh - gradients of exact attention over packed sequences
// on sm_100a (tcgen05 + TMEM + TMA).
//
//   P = exp(scale q.k - lse),  D_i = dO_i . o_i,  dS = P (dO.v - D),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K,
// dK and dV summed over the query heads of a KV head.
//
// Every output row is summed by one CTA in one order: no atomics, no 32-bit
// dQ in memory, and the same bits from every run. The price is that P and dS
// are formed twice, once for dK and dV and once for dQ (7 products of tile
// size instead of 5). The dense backward (bwd_sm100.cuh) forms them once and adds
// 32-bit dQ tiles in L2, in any order: 0.90 PFLOP/s of five products over 32768
// tokens, where this one has 0.67 (below) over shorter sequences.
//
// One CTA per item, one launch for both kinds:
//   key item   128 keys of one sequence and KV head. K and V stay; tiles of 128
//              rows (token, query head of the group) of Q and dO stream past:
//                S^T = K Q^T, dP^T = V dO^T   (lanes = keys)
//                dV += P^T dO, dK += dS^T Q   (A from TMEM)
//   row item   128 rows of one sequence and KV head. Q and dO stay; tiles of
//              128 keys of K and V stream past:
//                S = Q K^T, dP = dO V^T       (lanes = rows)
//                dQ += dS K                   (A from TMEM)
// Warps 0-7 form P and dS (thread = TMEM lane, warpgroup w = columns
// [64 w, 64 w + 64)); warp 8: TMA producer; warp 9: tcgen05 issuer; warp 10:
// finds the item, then brings the rows' statistics (key item) or means of the
// keys (row item). P and dS go back to TMEM as 16-bit pairs, each warpgroup's
// over its own columns.
//
// Rounding: P and dS to the inputs' type before their products, the outputs
// once; all sums and statistics in fp32.
//
// What bounds it: the tensor core with its issue, 80 cycles per 128 x 128 x 16
// product (cuBLAS takes about 84); a key item's step takes about 3700 cycles
// for 2560 of products, waiting for P's 128 x 128 exponentials (1024 cycles of
// MUFU), a row item's about 2600 for 1920. 16384 tokens in 5 sequences, 32 / 8
// heads of 128, bf16, causal: 2.48 ms at 1.74 GHz, 2.78 ms in passes in a row (the
// card's power cap), 0.67 PFLOP/s counting five products.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/blasst.h"
#include "attn_seq_sm100.cuh"
#include "ptx_sm100.cuh"

namespace blasst {

struct SeqBwdParams {
  void* dq;  // [Tq, Hq, D]
  void* dk;  // [Tk, Hkv, D]
  void* dv;  // [Tk, Hkv, D]
  const float2* stats;    // bf16: [Hkv][Tq][g] (-lse log2 e, D)
  const float* dsum;      // fp16: [Hkv][Tq][g] D,
  const uint32_t* sizes;  // [Hkv][Tq][g] sizes for dS' scale (SeqBwdScale),
  const float* lse;       // [Tq, Hq]
  const int* cu_q;
  const int* cu_k;
  const void* k;
  long long k_st, k_sh;
  int n_seq, Tq, Tk, Hq, Hkv, g;
  int rt;       // tokens per 128-row tile
  int n_key, n_row;  // places for items per KV head
  int causal;
  float scale, scale_log2;
  int* err;
  uint64_t timeout_ns;
};

// fp16 only: P (at most 1, but for the rounding of lse) is kept as 2^14 P, so that
// small P keep all their bits down to 2^-28 (dv of a key that only small weights
// touch is made of them), and dS as 2^k dS: |dS| <= 2 |dO_i| |v_j|, so with k from
// the largest rows of dO and v 2^k dS < 2^15 never overflows and uses the whole
// range. The largest are those of what is summed: for dQ the row of dO itself and
// the sequence's rows of v, for dK the sequence's rows of dO that see the keys. No
// other sequence has a part in it, nor has a large row in another row's dQ. Powers
// of two, undone in 32 bits at the end.
//
// A size is the upper half of |row|^2 as fp32, rounded up; 0 for rows that are not
// finite (their products are not either). sizes[hk][t][h]: the lower 16 bits are
// the size of the row of dO, the upper 16 of a sequence's first rows those of the
// largest row of v in a part of its keys (SeqSizeParts). Each is stored once, by one
// block: nothing to clear, no atomics (an atomic maximum per sequence cost a short
// call 2.5 us).
template <typename T>
struct SeqBwdType {
  static constexpr bool kScaled = SeqType<T>::kFormat == 0;
  static constexpr float kShift = kScaled ? 14.0f : 0.0f;
};

__device__ __forceinline__ uint32_t seq_size(float squares) {
  return squares < INFINITY ? (__float_as_uint(squares) + 0xffffu) >> 16 : 0u;
}

// k of 2^k dS from two sizes.
__device__ __forceinline__ int seq_ds_shift(uint32_t a, uint32_t b) {
  const float n = sqrtf(__uint_as_float(a << 16)) * sqrtf(__uint_as_float(b << 16));
  return n > 0.0f ? 13 - ilogbf(n) : 0;
}

// Sizes of v: a sequence's keys in parts of 64, or, where those are more than its
// rows, in as many times 64 as make them no more.
constexpr int kBwdRowsPerBlock = 64;
struct SeqSizeParts {
  int parts, tiles;  // of the sequence; of 64 keys in a part
};
__device__ __forceinline__ SeqSizeParts seq_size_parts(int kvlen, int qlen, int g) {
  const int tiles = (kvlen + kBwdRowsPerBlock - 1) / kBwdRowsPerBlock;
  const long long rows = static_cast<long long>(qlen) * g;
  if (tiles <= rows) return {tiles, 1};
  const int r = static_cast<int>(rows);
  const int each = (tiles + r - 1) / r;
  return {(tiles + each - 1) / each, each};
}

struct SeqBwdRowsParams {
  const void* o;
  const void* dout;
  const void* v;
  const float* lse;  // [Tq, Hq]
  float2* stats;     // bf16
  float* dsum;       // fp16
  uint32_t* sizes;
  const int* cu_q;
  const int* cu_k;
  long long o_st, o_sh, do_st, do_sh, v_st, v_sh;
  int n_seq, Tq, Tk, Hq, Hkv, g;
  int row_blocks;  // blocks over the query rows; those behind them take v
};

// Row pass: D_i of every row, with the scaled lse (bf16) or the row's size (fp16,
// where blocks behind those of the rows take the parts of v), laid out so that a
// tile's rows are contiguous. D / 8 lanes per row (16 bytes each), every warp all
// its rows' loads at once. Bound by memory: o and dO read once.
template <int D, typename T>
__global__ void __launch_bounds__(256) blasst_seq_bwd_rows_kernel(const SeqBwdRowsParams p) {
  ptx::grid_launch_dependents();     // (the pair kernel waits before it reads what is written here)
  constexpr bool SCALED = SeqBwdType<T>::kScaled;
  constexpr int LPR = D / 8;         // lanes per row
  constexpr int RPW = 32 / LPR;      // rows per warp
  constexpr int N = kBwdRowsPerBlock / (8 * RPW);
  const int hk = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, at = lane % LPR;
  const long long all = static_cast<long long>(p.Tq) * p.g;
  // the sum over a row's lanes, to all of them
  auto row_sum = [](float x) -> float {
#pragma unroll
    for (int d = LPR / 2; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
  };
  if (SCALED && static_cast<int>(blockIdx.x) >= p.row_blocks) {
    // ---- a part of v: its largest row ---------------------------------------
    const int place = static_cast<int>(blockIdx.x) - p.row_blocks;
    const int s = seq_of_place(p.cu_k, p.n_seq, p.Tk, kBwdRowsPerBlock, place, lane);
    if (s < 0) return;
    const SeqSpan q = seq_span(p.cu_q, p.cu_k, nullptr, 0, p.Tq, p.Tk, 1, s, nullptr);
    const int part = place - seq_place(p.cu_k, s, p.Tk, kBwdRowsPerBlock);
    if (q.qlen == 0) return;  // no rows: nobody reads it
    const SeqSizeParts parts = seq_size_parts(q.kvlen, q.qlen, p.g);
    if (part >= parts.parts) return;
    const long long keys = static_cast<long long>(parts.tiles) * kBwdRowsPerBlock;
    const int end = static_cast<int>(min(static_cast<long long>(q.kvlen), (part + 1) * keys));
    uint32_t most = 0;
#pragma unroll 4
    for (int r = static_cast<int>(part * keys) + warp * RPW; r < end; r += 8 * RPW) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r + sub < end)
        v = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + static_cast<long long>(q.k0 + r + sub) * p.v_st +
                                            hk * p.v_sh + at * 8);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float sq0 = 0.0f, sq1 = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a0, a1;
        seq_unpack2<T>(w[j], a0, a1);
        ptx::fma2(sq0, sq1, a0, a1, a0, a1, sq0, sq1);
      }
      most = max(most, seq_size(row_sum(sq0 + sq1)));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    __shared__ uint32_t of_warp[8];
    if (lane == 0) of_warp[warp] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < 8; ++i) most = max(most, of_warp[i]);
      reinterpret_cast<unsigned short*>(p.sizes + (static_cast<long long>(hk) * p.Tq + q.q0) * p.g + part)[1] =
          static_cast<unsigned short>(most);
    }
    return;
  }
  // ---- rows ------------------------------------------------------------------
  const long long block = blockIdx.x;
  // what belongs to no sequence is not read (it may hold anything)
  const uint32_t per = p.g;
  const long long begin = static_cast<long long>(max(p.cu_q[0], 0)) * per;
  const long long end = static_cast<long long>(min(p.cu_q[p.n_seq], p.Tq)) * per;
  uint4 av[N], bv[N];
  float lse[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const long long r = block * kBwdRowsPerBlock + (i * 8 + warp) * RPW + sub;
    av[i] = bv[i] = make_uint4(0u, 0u, 0u, 0u);
    lse[i] = 0.0f;
    if (r < begin || r >= end) continue;
    // (rows count below 2^38; within a KV head 32 bits hold tokens and heads)
    const long long t = all >> 32 ? r / per : static_cast<uint32_t>(r) / per;
    const int h = hk * p.g + static_cast<int>(r - t * per);
    av[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.dout) + t * p.do_st + h * p.do_sh + at * 8);
    bv[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.o) + t * p.o_st + h * p.o_sh + at * 8);
    if (!SCALED && at == 0) lse[i] = p.lse[t * p.Hq + h];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const long long r = block * kBwdRowsPerBlock + (i * 8 + warp) * RPW + sub;
    const uint32_t aw[4] = {av[i].x, av[i].y, av[i].z, av[i].w};
    const uint32_t bw[4] = {bv[i].x, bv[i].y, bv[i].z, bv[i].w};
    float dot0 = 0.0f, dot1 = 0.0f, sq0 = 0.0f, sq1 = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a0, a1, b0, b1;
      seq_unpack2<T>(aw[j], a0, a1);
      seq_unpack2<T>(bw[j], b0, b1);
      ptx::fma2(dot0, dot1, a0, a1, b0, b1, dot0, dot1);
      if (SCALED) ptx::fma2(sq0, sq1, a0, a1, a0, a1, sq0, sq1);
    }
    const float dot = row_sum(dot0 + dot1);
    const uint32_t size = SCALED ? seq_size(row_sum(sq0 + sq1)) : 0u;
    if (at != 0 || r < begin || r >= end) continue;
    const long long place = static_cast<long long>(hk) * all + r;
    if (SCALED) {
      p.dsum[place] = dot;
      *reinterpret_cast<unsigned short*>(p.sizes + place) = static_cast<unsigned short>(size);
    } else {
      p.stats[place] = make_float2(lse[i] == -INFINITY ? -INFINITY : lse[i] * -1.4426950408889634f, dot);
    }
  }
}

template <bool B>
struct SeqBool {
  static constexpr bool value = B;
};

template <int D>
struct SeqBwdCfg {
  static constexpr int NTHREADS = 384;
  // registers per thread, as in the forward
  static constexpr int REGS = 168, REGS_SOFT = 216, REGS_REST = 72;
  static constexpr int WARP_LOAD = 8, WARP_MMA = 9, WARP_ROWS = 10;
  static constexpr int BK = 128;
  static constexpr int DBOX = D / 64;
  static constexpr int BOX = 128 * 128;
  static constexpr int TILE = BOX * DBOX;
  // ring of the streamed tile that is read twice (Q, K) and of the other (dO, V)
  static constexpr int NS1 = D == 128 ? 3 : 4;
  static constexpr int NS2 = D == 128 ? 2 : 3;
  static constexpr int NST = 2;  // slots of row statistics
  static constexpr int OFF_A = 0;  // what stays: K, V or Q, dO
  static constexpr int OFF_R1 = 2 * TILE;
  static constexpr int OFF_R2 = OFF_R1 + NS1 * TILE;
  // key item: [NST][2][128] fp32 statistics; row item: [2][128] what the
  // roundings of dS lost, [3][D] means of the keys
  static constexpr int OFF_ST = OFF_R2 + NS2 * TILE;
  static constexpr int ST_BYTES = 1024 + (3 * D * 4 > 1024 ? 3 * D * 4 : 1024);
  static_assert(ST_BYTES >= NST * 1024, "statistics' slots");
  static constexpr int OFF_BAR = OFF_ST + ST_BYTES;
  static constexpr int B_A = 0;
  static constexpr int B_TAIL = 1;
  static constexpr int B_F1 = 2;
  static constexpr int B_E1 = B_F1 + NS1;
  static constexpr int B_F2 = B_E1 + NS1;
  static constexpr int B_E2 = B_F2 + NS2;
  static constexpr int B_S = B_E2 + NS2;   // S written
  static constexpr int B_P = B_S + 1;      // key item: P written; row item: S read (8 warps)
  static constexpr int B_DP = B_P + 1;     // [2] dP written
  static constexpr int B_DS = B_DP + 2;    // [2] dS written (8 warps)
  static constexpr int B_STF = B_DS + 2;   // [NST] statistics there
  static constexpr int B_STE = B_STF + NST;  // [NST] read (8 warps)
  static constexpr int B_ACC = B_STE + NST;
  static constexpr int B_DRAIN = B_ACC + 1;
  static constexpr int NBAR = B_DRAIN + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  // misc words: [0] tmem base, [1] abort, [3] always 0, [4..] the item
  static constexpr int OFF_ITEM = OFF_MISC + 16;
  static constexpr int OFF_SIZE = OFF_ITEM + 48;  // [9] largest sizes the warps found
  static constexpr int SMEM_BYTES = OFF_SIZE + 48;
  static constexpr int S_COL = 0;
  // key item: dP, dV, dK behind S; row item: dQ, then two dP
  static constexpr int K_DP = 128, K_DV = 256, K_DK = 384;
  static constexpr int R_DQ = 128, R_DP = 256;
  static constexpr int TMEM_COLS = 512;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

// The CTA's item. Tokens and keys count from the sequence's first.
struct SeqBwdItem {
  int kind;      // 0 none, 1 key item, 2 row item
  int hk, q0, qlen, k0, kvlen, off;
  int at;        // first key, or first token
  int first;     // key item: first token that is streamed
  int steps;     // streamed tiles
};

template <int D, typename T>
__global__ void __launch_bounds__(384, 1)
    blasst_seq_bwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmDO,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const SeqBwdParams p) {
  using C = SeqBwdCfg<D>;
  constexpr uint32_t IDESC_S = ptx::idesc_f32acc(SeqType<T>::kFormat, 128, 128, false);
  constexpr uint32_t IDESC_G = ptx::idesc_f32acc(SeqType<T>::kFormat, 128, D, true);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  const uint32_t sb = ptx::smem_u32(smem);
  volatile int* misc = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  volatile int* abort_flag = misc + 1;
  volatile int* itemw = reinterpret_cast<volatile int*>(smem + C::OFF_ITEM);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8 * i; };
  if ((sb & 1023u) != 0u) {  // uniform; the tiles need 1 KB alignment
    ptx::grid_wait();
    if (threadIdx.x == 0) seq_record_error(p.err, BLASST_EUNSUPPORTED);
    return;
  }

  // ---- the item: key items of all heads first, then row items -------------
  if (warp == C::WARP_ROWS) {
    const int n_keys = p.n_key * p.Hkv;
    const bool key = static_cast<int>(blockIdx.x) < n_keys;
    const int idx = key ? blockIdx.x : blockIdx.x - n_keys;
    const int per = key ? p.n_key : p.n_row;
    const int tile = key ? C::BK : p.rt, tokens = key ? p.Tk : p.Tq;
    const int* cu = key ? p.cu_k : p.cu_q;
    // longest first under a causal mask: the first keys, the last rows
    const int place = key ? idx % per : per - 1 - idx % per;
    // after a wait gave up, calls before blasst_check do nothing
    const bool live = !(p.err && *reinterpret_cast<volatile int*>(p.err) == BLASST_ETIMEOUT);
    const int s = live ? seq_of_place(cu, p.n_seq, tokens, tile, place, lane) : -1;
    SeqBwdItem it{};
    if (s >= 0) {
      const SeqSpan q = seq_span(p.cu_q, p.cu_k, nullptr, 0, p.Tq, p.Tk, p.rt, s, p.err);
      const int t = place - seq_place(cu, s, tokens, tile);
      if (t < (key ? (q.kvlen + C::BK - 1) / C::BK : q.tiles)) {
        it.hk = idx / per;
        it.q0 = q.q0;
        it.qlen = q.qlen;
        it.k0 = q.k0;
        it.kvlen = q.kvlen;
        it.off = q.off;
        it.at = t * tile;
        if (key) {
          it.kind = 1;
          // from the first token that sees a key of the tile: no row without
          // keys is ever streamed
          it.first = p.causal ? min(max(it.at - q.off, 0), q.qlen) : 0;
          it.steps = (q.qlen - it.first + p.rt - 1) / p.rt;
        } else {
          it.kind = 2;
          const int last = min(it.at + p.rt, q.qlen) - 1;
          const int keys = p.causal ? min(max(q.off + last + 1, 0), q.kvlen) : q.kvlen;
          it.steps = (keys + C::BK - 1) / C::BK;
        }
      }
    }
    if (lane == 0) {
      itemw[0] = it.kind;
      itemw[1] = it.hk;
      itemw[2] = it.q0;
      itemw[3] = it.qlen;
      itemw[4] = it.k0;
      itemw[5] = it.kvlen;
      itemw[6] = it.off;
      itemw[7] = it.at;
      itemw[8] = it.first;
      itemw[9] = it.steps;
    }
  }
  if (threadIdx.x == 0) {
    ptx::mbar_init(bar(C::B_A), 1);
    ptx::mbar_init(bar(C::B_TAIL), 1);
    for (int i = 0; i < C::NS1; ++i) {
      ptx::mbar_init(bar(C::B_F1 + i), 1);
      ptx::mbar_init(bar(C::B_E1 + i), 1);
    }
    for (int i = 0; i < C::NS2; ++i) {
      ptx::mbar_init(bar(C::B_F2 + i), 1);
      ptx::mbar_init(bar(C::B_E2 + i), 1);
    }
    ptx::mbar_init(bar(C::B_S), 1);
    ptx::mbar_init(bar(C::B_P), 8);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(C::B_DP + i), 1);
      ptx::mbar_init(bar(C::B_DS + i), 8);
    }
    for (int i = 0; i < C::NST; ++i) {
      ptx::mbar_init(bar(C::B_STF + i), 1);
      ptx::mbar_init(bar(C::B_STE + i), 8);
    }
    ptx::mbar_init(bar(C::B_ACC), 1);
    ptx::mbar_init(bar(C::B_DRAIN), 1);
    for (int i = 1; i < 4; ++i) misc[i] = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  SeqBwdItem it;
  it.kind = itemw[0];
  if (it.kind == 0) {  // uniform, nothing in flight
    ptx::grid_wait();    // (the row pass ends before this kernel does)
    return;
  }
  it.hk = itemw[1];
  it.q0 = itemw[2];
  it.qlen = itemw[3];
  it.k0 = itemw[4];
  it.kvlen = itemw[5];
  it.off = itemw[6];
  it.at = itemw[7];
  it.first = itemw[8];
  it.steps = itemw[9];
  const bool key = it.kind == 1;
  const int n = it.steps;
  const int box_rows = p.g * p.rt;
  if (warp == C::WARP_MMA) {
    ptx::tmem_alloc(ptx::smem_u32(const_cast<int*>(misc)), C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  if (key && box_rows < 128) {
    // rows of a streamed tile that no copy writes: contracted over, so 0
    for (int s = 0; s < C::NS1 + C::NS2; ++s)
      for (int x = 0; x < C::DBOX; ++x)
        for (int i = box_rows * 8 + threadIdx.x; i < 128 * 8; i += C::NTHREADS)
          *reinterpret_cast<uint4*>(smem + C::OFF_R1 + s * C::TILE + x * C::BOX + i * 16) =
              make_uint4(0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  auto fail = [&]() {
    *abort_flag = 1;
    seq_record_error(p.err, BLASST_ETIMEOUT);
  };
  auto warp_wait = [&](uint32_t b, uint32_t parity) -> bool {
    bool r = true;
    if (lane == 0) r = ptx::mbar_wait(b, parity, abort_flag, p.timeout_ns);
    return __shfl_sync(0xffffffffu, r ? 1 : 0, 0) != 0;
  };
  ptx::grid_wait();  // the rows' statistics (the set-up ran beside their pass)
  // dS = (2^shift P) (c dP - c D) = 2^k P (dP - D)
  float c = 1.0f;  // (a power of two; 2^-k is taken from it at the end)
  constexpr bool SCALED = SeqBwdType<T>::kScaled;
  constexpr float SHIFT = SeqBwdType<T>::kShift;
  auto seq_row_of = [&]() -> long long { return (static_cast<long long>(it.hk) * p.Tq + it.q0) * p.g; };  // the sequence's first
  auto set_scale = [&](uint32_t of_do, uint32_t of_v) {
    c = exp2f(static_cast<float>(seq_ds_shift(of_do, of_v)) - SHIFT);
  };
  // the sequence's largest row of v, to all lanes
  auto size_of_v = [&]() -> uint32_t {
    const int parts = seq_size_parts(it.kvlen, it.qlen, p.g).parts;
    uint32_t most = 0;
    for (int i = lane; i < parts; i += 32) most = max(most, p.sizes[seq_row_of() + i] >> 16);
    return __reduce_max_sync(0xffffffffu, most);
  };
  // key item: from the largest row of dO that is streamed, found by the warps that
  // need it (0-7, and 10) while the first tiles are on their way: 4 bytes per row
  // beside the 4 D that the row's streaming takes
  auto key_scale = [&]() {
    if (!SCALED || n == 0) return;
    const int group = warp == C::WARP_ROWS ? 8 : warp;
    const long long begin = seq_row_of() + static_cast<long long>(it.first) * p.g;
    const long long end = seq_row_of() + static_cast<long long>(it.qlen) * p.g;
    uint32_t most = 0;
    // four at a time, from the boundary before the first on (the workspace goes on behind the last)
#pragma unroll 4
    for (long long r = (begin & ~3ll) + 4 * (group * 32 + lane); r < end; r += 4 * 9 * 32) {
      const uint4 w = *reinterpret_cast<const uint4*>(p.sizes + r);
      if (r >= begin) most = max(most, w.x & 0xffffu);
      if (r + 1 >= begin && r + 1 < end) most = max(most, w.y & 0xffffu);
      if (r + 2 >= begin && r + 2 < end) most = max(most, w.z & 0xffffu);
      if (r + 3 >= begin && r + 3 < end) most = max(most, w.w & 0xffffu);
    }
    const uint32_t of_v = size_of_v();
    most = __reduce_max_sync(0xffffffffu, most);
    volatile uint32_t* part = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_SIZE);
    if (lane == 0) part[group] = most;
    ptx::named_bar_sync(1, 9 * 32);
#pragma unroll
    for (int i = 0; i < 9; ++i) most = max(most, part[i]);
    set_scale(most, of_v);
  };

  if (warp >= 8) {
    ptx::reg_give<C::REGS_REST>();
    if (warp == C::WARP_LOAD) {
      // ======================= TMA producer ==================================
      // rows (key item: tokens; row item: keys) of a streamed tile, and the
      // rows of each that count
      const CUtensorMap* a1 = key ? &tmK : &tmQ;
      const CUtensorMap* a2 = key ? &tmV : &tmDO;
      const CUtensorMap* s1 = key ? &tmQ : &tmK;
      const CUtensorMap* s2 = key ? &tmDO : &tmV;
      const int a_rows = key ? C::BK : box_rows, s_rows = key ? box_rows : C::BK;
      auto load = [&](const CUtensorMap* tm, bool of_keys, uint32_t dst, int row, uint32_t b) {
#pragma unroll
        for (int x = 0; x < C::DBOX; ++x) {
          if (of_keys) ptx::tma_load_4d(dst + x * C::BOX, tm, x * 64, it.k0 + row, it.hk, 0, b);
          else ptx::tma_load_4d(dst + x * C::BOX, tm, x * 64, 0, it.q0 + row, it.hk, b);
        }
      };
      bool ok = true;
      bool a_sent = false;
      uint32_t tails = 0, in1 = 0, in2 = 0;  // loads whose full barrier the copy itself completes
      bool tail_open = false;
      for (int i = 0; i < n && ok; ++i) {
        const int row = key ? it.first + i * p.rt : i * C::BK;
        const int valid = key ? min(p.rt, it.qlen - row) * p.g : min(C::BK, it.kvlen - row);
        const bool tail = valid < s_rows;
#pragma unroll 1
        for (int w = 0; w < 2 && ok; ++w) {
          const uint32_t slots = w ? C::NS2 : C::NS1;
          const uint32_t slot = static_cast<uint32_t>(i) % slots, turn = static_cast<uint32_t>(i) / slots;
          const uint32_t full = bar((w ? C::B_F2 : C::B_F1) + slot);
          const int off = (w ? C::OFF_R2 : C::OFF_R1) + static_cast<int>(slot) * C::TILE;
          // rows behind the sequence's end may hold anything, and 0 x NaN is
          // NaN: what is contracted over is cleared (V is not, its products
          // are replaced)
          const bool clear = tail && (key || w == 0);
          const uint32_t fb = clear ? bar(C::B_TAIL) : full;
          if (lane == 0) {
            if (turn > 0)
              ok = ptx::mbar_wait(bar((w ? C::B_E2 : C::B_E1) + slot), (turn - 1) & 1, abort_flag,
                                  p.timeout_ns);
            if (ok) {
              if (i == 0 && w == 0) {
                ptx::mbar_arrive_expect_tx(bar(C::B_A), 2 * C::DBOX * a_rows * 128);
                load(a1, key, sb + C::OFF_A, it.at, bar(C::B_A));
              }
              ptx::mbar_arrive_expect_tx(fb, C::DBOX * s_rows * 128);
              load(w ? s2 : s1, !key, sb + off, row, fb);
              if (i == 0 && w == 0) load(a2, key, sb + C::OFF_A + C::TILE, it.at, bar(C::B_A));
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          a_sent = true;
          if (w) in2 = i + 1;
          else in1 = i + 1;
          if (clear) {
            tail_open = true;
            ok = warp_wait(bar(C::B_TAIL), tails & 1);
            if (!ok) break;
            ++tails;
            tail_open = false;
            for (int u = valid * 8 + lane; u < 128 * 8; u += 32)
#pragma unroll
              for (int x = 0; x < C::DBOX; ++x)
                *reinterpret_cast<uint4*>(smem + off + x * C::BOX + u * 16) = make_uint4(0u, 0u, 0u, 0u);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(full);
          }
        }
      }
      if (!ok && lane == 0) {
        fail();
        // copies in flight land before the CTA exits (1 ms each is ample)
        const uint64_t drain_ns = p.timeout_ns < 1000000ull ? p.timeout_ns : 1000000ull;
        if (a_sent) ptx::mbar_wait(bar(C::B_A), 0, &misc[3], drain_ns);
        if (tail_open) ptx::mbar_wait(bar(C::B_TAIL), tails & 1, &misc[3], drain_ns);
        for (uint32_t k = in1 < C::NS1 ? 0 : in1 - C::NS1; k < in1; ++k)
          ptx::mbar_wait(bar(C::B_F1 + k % C::NS1), (k / C::NS1) & 1, &misc[3], drain_ns);
        for (uint32_t k = in2 < C::NS2 ? 0 : in2 - C::NS2; k < in2; ++k)
          ptx::mbar_wait(bar(C::B_F2 + k % C::NS2), (k / C::NS2) & 1, &misc[3], drain_ns);
      }
    } else if (warp == C::WARP_MMA) {
      // ======================= tcgen05 issuer ================================
      if (n > 0 && ptx::elect_one()) {
        const uint64_t a_desc = ptx::sw128_desc(sb + C::OFF_A, 16, 1024);
        const uint64_t b1_desc = ptx::sw128_desc(sb + C::OFF_R1, 16, 1024);
        const uint64_t b2_desc = ptx::sw128_desc(sb + C::OFF_R2, 16, 1024);
        const uint64_t g1_desc = ptx::sw128_desc(sb + C::OFF_R1, C::BOX, 1024);
        const uint64_t g2_desc = ptx::sw128_desc(sb + C::OFF_R2, C::BOX, 1024);
        constexpr uint64_t TS = C::TILE >> 4;
        auto wait = [&](int b, uint32_t parity) -> bool {
          return ptx::mbar_wait(bar(b), parity, abort_flag, p.timeout_ns);
        };
        // 128 x 128 products of what stays and a streamed tile (K-major both)
        auto score = [&](uint32_t d_tm, uint64_t a, uint64_t b) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t o = static_cast<uint64_t>(((kk >> 2) * C::BOX + (kk & 3) * 32) >> 4);
            ptx::mma_ss(d_tm, a + o, b + o, IDESC_S, kk > 0 ? 1u : 0u);
          }
        };
        // 128 x D: 16-bit pairs in TMEM (each warpgroup's over its columns)
        // times a streamed tile
        auto grad = [&](uint32_t d_tm, uint32_t a_tm, uint64_t b, bool add) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            ptx::mma_ts(d_tm, a_tm + (kk >> 2) * 64 + (kk & 3) * 8,
                        b + static_cast<uint64_t>(kk * (2048 >> 4)), IDESC_G,
                        add || kk > 0 ? 1u : 0u);
        };
        auto issue_s = [&](int i) -> bool {
          const uint32_t slot = static_cast<uint32_t>(i) % C::NS1, turn = static_cast<uint32_t>(i) / C::NS1;
          if (!wait(C::B_F1 + slot, turn & 1)) return false;
          ptx::tc_fence_after();
          score(tmem + C::S_COL, a_desc, b1_desc + slot * TS);
          ptx::mma_commit(bar(C::B_S));
          return true;
        };
        auto issue_dp = [&](int i) -> bool {
          const uint32_t slot = static_cast<uint32_t>(i) % C::NS2, turn = static_cast<uint32_t>(i) / C::NS2;
          if (!wait(C::B_F2 + slot, turn & 1)) return false;
          ptx::tc_fence_after();
          score(tmem + (key ? C::K_DP : C::R_DP + (i & 1) * 128), a_desc + TS, b2_desc + slot * TS);
          ptx::mma_commit(bar(C::B_DP + (i & 1)));
          if (!key) ptx::mma_commit(bar(C::B_E2 + slot));
          return true;
        };
        bool ok = wait(C::B_A, 0);
        ok = ok && issue_s(0) && issue_dp(0);
        for (int i = 0; i < n && ok; ++i) {
          const uint32_t s1 = static_cast<uint32_t>(i) % C::NS1, s2 = static_cast<uint32_t>(i) % C::NS2;
          if (key) {
            // dV(i), S(i+1), dK(i), dP(i+1): while dS(i) is formed the tensor
            // core does the first two, while P(i+1) is formed the others
            ok = wait(C::B_P, i & 1);
            if (!ok) break;
            ptx::tc_fence_after();
            grad(tmem + C::K_DV, tmem + C::S_COL, g2_desc + s2 * TS, i > 0);
            ptx::mma_commit(bar(C::B_E2 + s2));
            if (i + 1 < n) ok = issue_s(i + 1);  // over P(i), which dV(i) has read by then
            ok = ok && wait(C::B_DS + (i & 1), (i >> 1) & 1);
            if (!ok) break;
            ptx::tc_fence_after();
            grad(tmem + C::K_DK, tmem + C::K_DP, g1_desc + s1 * TS, i > 0);
            ptx::mma_commit(bar(C::B_E1 + s1));
            if (i + 1 < n) ok = issue_dp(i + 1);
          } else {
            if (i + 1 < n) {
              ok = wait(C::B_P, i & 1);
              ok = ok && issue_s(i + 1) && issue_dp(i + 1);
            }
            ok = ok && wait(C::B_DS + (i & 1), (i >> 1) & 1);
            if (!ok) break;
            ptx::tc_fence_after();
            grad(tmem + C::R_DQ, tmem + C::R_DP + (i & 1) * 128, g1_desc + s1 * TS, i > 0);
            ptx::mma_commit(bar(C::B_E1 + s1));
          }
        }
        ptx::mma_commit(bar(C::B_ACC));
        if (!ok) fail();
        // every product has completed before TMEM is freed
        ptx::mma_commit(bar(C::B_DRAIN));
        ptx::mbar_wait(bar(C::B_DRAIN), 0, &misc[3], p.timeout_ns);
      }
    } else if (warp == C::WARP_ROWS && key) {
      // ======================= statistics of the streamed rows ===============
      bool ok = true;
      int of_lse[4];  // this lane's rows of a tile in lse
#pragma unroll
      for (int u = 0; u < 4; ++u) of_lse[u] = (lane + 32 * u) / p.g * p.Hq + it.hk * p.g + (lane + 32 * u) % p.g;
      for (int i = 0; i < n && ok; ++i) {
        const int slot = i % C::NST;
        const int tok = it.first + i * p.rt;
        const int valid = min(p.rt, it.qlen - tok) * p.g;
        float2 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = lane + 32 * u;
          v[u] = make_float2(-INFINITY, 0.0f);
          if (r >= valid) continue;
          const long long place = seq_row_of() + static_cast<long long>(tok) * p.g + r;
          if constexpr (SCALED) v[u] = make_float2(p.lse[static_cast<long long>(it.q0 + tok) * p.Hq + of_lse[u]], p.dsum[place]);
          else v[u] = p.stats[place];
        }
        if (i == 0) key_scale();
        if (i >= C::NST) ok = warp_wait(bar(C::B_STE + slot), (i / C::NST - 1) & 1);
        if (!ok) break;
        float* st = reinterpret_cast<float*>(smem + C::OFF_ST + slot * 1024);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          st[lane + 32 * u] =
              SCALED && v[u].x != -INFINITY ? fmaf(v[u].x, -1.4426950408889634f, SHIFT) : v[u].x;
          st[128 + lane + 32 * u] = -v[u].y * c;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_STF + slot));
      }
      if (!ok && lane == 0) fail();
    } else if (warp == C::WARP_ROWS && n > 0) {
      // ======================= means of the keys =============================
      // Of up to 32 keys that every row of the item sees; at a sequence's start,
      // where the first row sees few, also of the first 4 and 16 for the rows
      // that see those. Each is drawn towards 0 by what a mean of so few is off
      // (Stein: by V / n of |mean|^2, V the keys' variance); of one key nothing
      // is known (taken for the mean it made dQ of 40 causal tokens worse than
      // without any: error 2.8e-3 where two roundings make 2.4e-3). Against no
      // means, 2000 causal tokens of 8 / 2 heads of 128, bf16, dQ's error in units of
      // its own rounding: keys of mean 0 1.47 both ways, of 0.5 deviations 1.67 for
      // 1.74, of 2 3.2 for 3.8, of 8 11.3 for 13.9 (the rest is o's rounding, in D);
      // it takes 6 to 7 % of the kernel's time.
      const int m = p.causal ? min(it.off + it.at + 1, it.kvlen) : it.kvlen;
      const int most = p.causal ? min(it.off + min(it.at + p.rt, it.qlen), it.kvlen) : it.kvlen;
      // four columns per lane, and of d = 64 two keys at a time
      constexpr int LPK = D / 4, KP = 32 / LPK;
      const int sub = lane / LPK, col = lane % LPK * 4;
      const T* base = static_cast<const T*>(p.k) + static_cast<long long>(it.k0) * p.k_st + it.hk * p.k_sh + col;
      // `count` keys, evenly over the first `over`
      auto mean_of = [&](int level, int count, int over) {
        float sum[4] = {0.f, 0.f, 0.f, 0.f}, squares = 0.0f, of_mean = 0.0f;
#pragma unroll 1
        for (int i0 = sub; i0 < count; i0 += 4 * KP) {
          uint2 w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * KP;
            const T* at = base + (over <= 32 ? i : (static_cast<long long>(i) * over) >> 5) * p.k_st;
            w[j] = i < count ? *reinterpret_cast<const uint2*>(at) : make_uint2(0u, 0u);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x[4];
            seq_unpack2<T>(w[j].x, x[0], x[1]);
            seq_unpack2<T>(w[j].y, x[2], x[3]);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              sum[v] += x[v];
              squares = fmaf(x[v], x[v], squares);
            }
          }
        }
        __syncwarp();
        const float keys = static_cast<float>(max(count, 2));
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if (KP == 2) sum[v] += __shfl_xor_sync(0xffffffffu, sum[v], 16);
          sum[v] /= keys;
          of_mean = fmaf(sum[v], sum[v], of_mean);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          squares += __shfl_xor_sync(0xffffffffu, squares, d);
          of_mean += __shfl_xor_sync(0xffffffffu, of_mean, d);
        }
        of_mean /= static_cast<float>(KP);
        const float variance = fmaxf(squares - keys * of_mean, 0.0f) / (keys - 1.0f);
        const float part = count > 1 && of_mean > 0.0f ? fmaxf(1.0f - variance / (keys * of_mean), 0.0f) : 0.0f;
        if (sub == 0)
          *reinterpret_cast<float4*>(smem + C::OFF_ST + 1024 + (level * D + col) * 4) =
              part > 0.0f ? make_float4(sum[0] * part, sum[1] * part, sum[2] * part, sum[3] * part)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
      };
#pragma unroll 1
      for (int level = 0; level < 3; ++level) {
        const int count = level == 0 ? max(min(m, 32), 0) : level == 1 ? 4 : 16;
        if (level == 0 || (m < count && count <= most)) mean_of(level, count, level == 0 ? m : count);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(C::B_STF));
    }
  } else {
    ptx::reg_take<C::REGS_SOFT>();
    // (compiled once per kind of item)
    auto compute = [&](auto kind) {
      constexpr bool key = decltype(kind)::value;
      // ======================= P and dS ========================================
      if (key) key_scale();
      const int wg = warp >> 2;
      const int row = (warp & 3) * 32 + lane;  // TMEM lane
      const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t s_tm = tmem + lane_base + C::S_COL + wg * 64;
      const float sl2 = p.scale_log2;
      bool ok = true;
      volatile float* all = reinterpret_cast<volatile float*>(smem + C::OFF_ST);
      // row item: the lane's token and statistics
      const int tok = it.at + row / p.g;
      const bool exists = key ? it.at + row < it.kvlen : row < box_rows && tok < it.qlen;
      float nl2 = -INFINITY, dcol = 0.0f;
      int limit = 0, least = 0;
      if (!key) {
        const uint32_t of_v = SCALED && n > 0 ? size_of_v() : 0u;
        if (exists) {
          const long long place = seq_row_of() + static_cast<long long>(it.at) * p.g + row;
          if constexpr (SCALED) {
            const float lse = p.lse[static_cast<long long>(it.q0 + tok) * p.Hq + it.hk * p.g + row % p.g];
            if (n > 0) set_scale(p.sizes[place] & 0xffffu, of_v);
            nl2 = lse == -INFINITY ? -INFINITY : fmaf(lse, -1.4426950408889634f, SHIFT);
            dcol = -p.dsum[place] * c;
          } else {
            const float2 v = p.stats[place];
            nl2 = v.x;
            dcol = -v.y * c;
          }
        }
        limit = p.causal ? min(it.off + tok + 1, it.kvlen) : it.kvlen;
        least = p.causal ? min(it.off + it.at + 1, it.kvlen) : it.kvlen;
        // the mean of the most keys that the lane's row sees for certain; kept in
        // shared memory meanwhile (the loop has no register to spare)
        all[wg * 128 + row] = least < 16 && limit >= 16 ? 2.0f : least < 4 && limit >= 4 ? 1.0f : 0.0f;
      }
      // Row item: dQ = scale (sum_j r_ij k_j + (sum_j dS_ij - r_ij) kappa), r = dS
      // rounded, kappa a mean of the keys. What all keys have in common (often
      // large) cancels in the exact sum, as sum_j dS_ij is 0 but for o's own
      // rounding; r's errors do not cancel it and are kept from it this way.
      float lost = 0.0f;
      float pv[64];
      // the lane's visible columns of tile i: [lo, hi), relative to the warpgroup's
      auto columns = [&](int i, int& lo, int& hi) -> bool {
        lo = 0;
        hi = 64;
        if (key) {
          if (!p.causal) return false;
          const int first = it.first + i * p.rt + it.off;  // key the tile's first token sees last
          lo = max(it.at + row - first, 0) * p.g - wg * 64;
          return it.at + C::BK - 1 > first;
        }
        const int col0 = i * C::BK;
        hi = limit - col0 - wg * 64;
        return col0 + C::BK > least;
      };
      auto form_p = [&](int i) -> bool {
        if (!warp_wait(bar(C::B_S), i & 1)) return false;
        if (key && !warp_wait(bar(C::B_STF + i % C::NST), (i / C::NST) & 1)) return false;
        ptx::tc_fence_after();
        uint32_t sv[64];
        ptx::tmem_ld32p(s_tm, sv);
        ptx::tmem_ld32p(s_tm + 32, sv + 32);
        ptx::tmem_wait_ld();
        if (!key) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(C::B_P));
        }
        const float4* st = reinterpret_cast<const float4*>(smem + C::OFF_ST + (i % C::NST) * 1024) + wg * 16;
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          float4 a = make_float4(nl2, nl2, nl2, nl2);
          if (key) a = st[j / 4];
          float x0, x1, x2, x3;
          ptx::fma2(x0, x1, __uint_as_float(sv[j]), __uint_as_float(sv[j + 1]), sl2, sl2, a.x, a.y);
          ptx::fma2(x2, x3, __uint_as_float(sv[j + 2]), __uint_as_float(sv[j + 3]), sl2, sl2, a.z, a.w);
          pv[j] = ptx::ex2(x0);
          pv[j + 1] = ptx::ex2(x1);
          pv[j + 2] = ptx::ex2(x2);
          pv[j + 3] = ptx::ex2(x3);
        }
        int lo, hi;
        if (columns(i, lo, hi)) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (j < lo || j >= hi) pv[j] = 0.0f;
        }
        if (key) {
          uint32_t pk[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) pk[j] = seq_pack2<T>(pv[2 * j], pv[2 * j + 1]);
          ptx::tmem_st32(s_tm, pk);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(C::B_P));
        }
        return true;
      };
      auto form_ds = [&](int i) -> bool {
        if (!warp_wait(bar(C::B_DP + (i & 1)), (i >> 1) & 1)) return false;
        ptx::tc_fence_after();
        const uint32_t dp_tm =
            tmem + lane_base + (key ? C::K_DP : C::R_DP + (i & 1) * 128) + wg * 64;
        uint32_t dp[64];
        ptx::tmem_ld32p(dp_tm, dp);
        ptx::tmem_ld32p(dp_tm + 32, dp + 32);
        ptx::tmem_wait_ld();
        const float4* st =
            reinterpret_cast<const float4*>(smem + C::OFF_ST + (i % C::NST) * 1024 + 512) + wg * 16;
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          float4 a = make_float4(dcol, dcol, dcol, dcol);
          if (key) a = st[j / 4];
          float x[4];
          ptx::fma2(x[0], x[1], __uint_as_float(dp[j]), __uint_as_float(dp[j + 1]), c, c, a.x, a.y);
          ptx::fma2(x[2], x[3], __uint_as_float(dp[j + 2]), __uint_as_float(dp[j + 3]), c, c, a.z, a.w);
          ptx::mul2(pv[j], pv[j + 1], x[0], x[1], pv[j], pv[j + 1]);
          ptx::mul2(pv[j + 2], pv[j + 3], x[2], x[3], pv[j + 2], pv[j + 3]);
        }
        int lo, hi;
        if (columns(i, lo, hi)) {  // a masked place may hold anything: 0, whatever dP is
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (j < lo || j >= hi) pv[j] = 0.0f;
        }
        uint32_t pk[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) pk[j] = seq_pack2<T>(pv[2 * j], pv[2 * j + 1]);
        ptx::tmem_st32(dp_tm, pk);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(bar(C::B_DS + (i & 1)));
          if (key) ptx::mbar_arrive(bar(C::B_STE + i % C::NST));
        }
        if (!key) {
          // (while S of the next tile is awaited)
          float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float r0, r1;
            seq_unpack2<T>(pk[j], r0, r1);
            ptx::fma2(r0, r1, r0, r1, -1.0f, -1.0f, pv[2 * j], pv[2 * j + 1]);
            const int a = 2 * (j & 1);
            ptx::add2(t[a], t[a + 1], t[a], t[a + 1], r0, r1);
          }
          lost += (t[0] + t[1]) + (t[2] + t[3]);
        }
        return true;
      };
      if (n > 0) ok = form_p(0);
      for (int i = 0; i < n && ok; ++i) {
        ok = form_ds(i);
        if (ok && i + 1 < n) ok = form_p(i + 1);
      }
      if (ok && n > 0) ok = warp_wait(bar(C::B_ACC), 0);
      float common = 0.0f;  // both warpgroups' `lost` of the lane's row
      const float* mean = reinterpret_cast<const float*>(smem + C::OFF_ST + 1024);
      if (!key && ok && n > 0) {
        mean += static_cast<int>(all[wg * 128 + row]) * D;
        all[wg * 128 + row] = lost;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_STE));
        ok = warp_wait(bar(C::B_STE), 0) && warp_wait(bar(C::B_STF), 0);
        if (ok) common = all[row] + all[128 + row];
      }
      ok = ok && *abort_flag == 0;
      ok = __all_sync(0xffffffffu, ok) != 0;
      if (!ok) {
        fail();
      } else {
        ptx::tc_fence_after();
        // key item: warpgroup 0 writes dV, 1 writes dK; row item: half of the
        // columns of dQ each
        const int chunks = key ? D / 32 : D / 64;
        const int c0 = key ? 0 : wg * (D / 64);
        const uint32_t acc = tmem + lane_base + (key ? (wg ? C::K_DK : C::K_DV) : C::R_DQ);
        const float f = (key && wg == 0 ? 1.0f : p.scale / c) * exp2f(-SHIFT);
        T* out;
        if (key) out = static_cast<T*>(wg ? p.dk : p.dv) +
                       (static_cast<long long>(itemw[4] + it.at + row) * p.Hkv + itemw[1]) * D;
        else out = static_cast<T*>(p.dq) +
                   (static_cast<long long>(itemw[2] + tok) * p.Hq + itemw[1] * p.g + row % p.g) * D;
#pragma unroll 1
        for (int k = c0; k < c0 + chunks; ++k) {
          uint32_t r[32];
          if (n > 0) {
            ptx::tmem_ld32(acc + 32 * k, r);
            ptx::tmem_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = 0u;
          }
          if (!key && n > 0) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              r[j] = __float_as_uint(fmaf(common, mean[32 * k + j], __uint_as_float(r[j])));
          }
          if (exists) {
            uint4* dst = reinterpret_cast<uint4*>(out + 32 * k);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int u = 0; u < 4; ++u)
                w[u] = seq_pack2<T>(__uint_as_float(r[8 * j + 2 * u]) * f,
                                    __uint_as_float(r[8 * j + 2 * u + 1]) * f);
              dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
    };
    if (key) compute(SeqBool<true>{});
    else compute(SeqBool<false>{});
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == C::WARP_MMA) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace blasst
