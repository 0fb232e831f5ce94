// attn_seq_sm100.cuh - exact attention over sequences of different lengths on
// sm_100a (tcgen05 + TMEM + TMA): prompts packed one behind the other, or new
// tokens (a chunk or a single one per sequence) against a paged KV cache.
//
// o_i = sum_j p_ij v_j / sum_j p_ij, p_ij = exp(scale q_i . k_j - m_i) over
// the keys j the mask leaves, one pass over the keys with a running reference
// m and sum l per row; lse_i = m + ln l. A row without keys gets o = 0,
// lse = -inf.
//
// A tile is 128 rows, each one (token, query head of one KV head's group):
// g = Hq / Hkv heads of floor(128 / g) tokens. All heads of a group share
// every K and V tile, and the causal diagonal crosses 128 / g tokens only. A
// CTA runs two streams of (S = Q K^T, softmax, O += P V), one softmax
// warpgroup each, so that the tensor core works on one stream while the other
// takes its exponentials:
//   two tiles  (more than 128 rows left): stream s owns rows tile s; both read
//              each K and V block once it is in shared memory;
//   one tile   (up to 128 rows, e.g. single tokens): both streams own the same
//              rows and take the even and the odd key blocks; their sums are
//              joined from TMEM at the end;
//   few rows   (one tile of up to 32 rows): the rows are repeated in the four
//              quarters of the TMEM lanes and quarter i takes the keys
//              [32 i, 32 i + 32) of a block (P is 0 elsewhere), so that all
//              four warps of a stream take exponentials; their sums are joined
//              through shared memory at the end. With one warp's 128 columns a
//              block took 2800 cycles of that warp and a step of single tokens
//              was bound by it (855 us for 4.3 GB of cached keys and values).
//              In a kernel of its own (FEW, which takes any item): beside the
//              others' block loop it made the compiler spill there (3.5 -> 6.2
//              ms for 32768 prompt tokens of 32 heads).
// Warps 0-3, 4-7: softmax of stream 0, 1 (thread = row = TMEM lane); warps 8
// and 11: TMA producers of Q and K, and of V; warp 9: tcgen05 issuer; warp 10:
// finds the CTA's items and hands the others one record each (warps 8-11 give
// registers to the softmax warps). TMEM: S0, S1 (fp32, 128 columns; P as
// 16-bit pairs over the first 64 of the same columns once S is in registers),
// O0, O1.
//
// Work: either whole items (sequence, KV head, tile), the last tiles of a head
// first (enough tiles to fill the GPU several times), which a resident grid
// takes one after the other from a list, so that one's output and the next
// one's loads overlap (32768 prompt tokens: 2.84 -> 2.74 ms over a CTA per
// item; results do not depend on who takes which); or a resident
// grid that cuts the list of all key blocks of all items into equal ranges
// ("shared list"), or, where that list is short, gives every CTA one piece of
// one item: an item cut by a range's or piece's end leaves fp32 partials,
// joined by seq_join_kernel in their order, so results do not depend on timing.
//
// Rounding: scores, the softmax's statistics, O and partials are fp32; P is
// rounded to the inputs' type, which the tensor core takes next to V (fp16: the
// reference lies 2^7 under the row's maximum for its range, SeqType), and
// o once at the end.
//
// What bounds it ("cool": single passes at 1.7 GHz or more; passes in a row run at
// the card's power cap). Long prompts: the tensor core with its issue, about 95
// cycles per 128 x 128 x 16 product beside the softmax's TMEM traffic (64 ideal;
// 32768 prompt tokens of 32 / 8 heads of 128, bf16: 2.76 ms cool, 1.13 PFLOP/s;
// 3.20 ms in a row, 0.97). Heads of 64: the exponentials with the same (14250
// tokens in two prompts of 64 / 8 heads, causal: 1.53 ms, where 16 exponentials a
// cycle take 0.75 and the products 0.52). Single tokens: memory (16 x 65536 cached
// tokens of 8 KV heads of 128: 650-740 us by how the pages lie, 0.90-0.97 of a
// copy's rate). Short calls: latency (511 tokens in 5 prompts: 13 us on the GPU, 2
// of set-up, 1.5 to find the item, 1.5 for the first loads).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/blasst.h"
#include "ptx_sm100.cuh"

namespace blasst {

struct SeqAttnParams {
  void* o;     // [Tq, Hq, D]
  float* lse;  // [Tq, Hq]
  const int* cu_q;
  const int* cu_k;     // packed keys; null with a page table
  const int* kv_lens;  // with a page table
  const int* table;
  long long table_stride;
  int table_width;
  int page_size, n_pages;
  // keys per TMA box, a power of two: 128, or the largest that divides page_size
  int chunk_log2;
  int n_seq, Tq, Tk, Hq, Hkv, g;
  int rt;        // tokens per 128-row tile
  int rt_few;    // tokens per 32 rows (0: a group is larger)
  int it_tok;    // tokens per item: rt (the kernel for few rows) or 2 rt
  int n_tiles;   // places for items per KV head (whole items); 0: shared list
  int* next;     // whole items: how many the CTAs took behind their first; null: one item per CTA
  int causal;
  float scale_log2;
  float* part_o;    // [2 * grid][256][D]
  float* part_lse;  // [2 * grid][256], log2 units
  int4* part_desc;  // [grid][2]
  int* err;
  uint64_t timeout_ns;
};

// One sequence's place in q and in the keys, read from the device arrays and
// clamped to the tensors (a clamp is reported: BLASST_EINDEX).
struct SeqSpan {
  int q0, qlen, k0, kvlen, off, tiles;
};

// `err`: the two device error words. An index error has one of its own: it must
// neither stop other calls, as a wait that gave up does, nor hide one.
__device__ __forceinline__ void seq_record_error(int* err, int code) {
  if (err) atomicCAS(code == BLASST_EINDEX ? err + 1 : err, 0, code);
}

__device__ __forceinline__ SeqSpan seq_span(const int* cu_q, const int* cu_k, const int* kv_lens,
                                            int kv_cap, int Tq, int Tk, int tile_tokens, int s,
                                            int* err) {
  SeqSpan r;
  const int q0 = cu_q[s], q1 = cu_q[s + 1];
  r.q0 = min(max(q0, 0), Tq);
  r.qlen = min(max(q1, r.q0), Tq) - r.q0;
  bool bad = q0 < 0 || q1 < q0 || q1 > Tq;
  if (cu_k) {
    const int a = cu_k[s], b = cu_k[s + 1];
    r.k0 = min(max(a, 0), Tk);
    r.kvlen = min(max(b, r.k0), Tk) - r.k0;
    bad = bad || a < 0 || b < a || b > Tk;
  } else {
    const int n = kv_lens[s];
    r.k0 = 0;
    r.kvlen = min(max(n, 0), kv_cap);
    bad = bad || n != r.kvlen;
  }
  if (bad) seq_record_error(err, BLASST_EINDEX);
  r.off = r.kvlen - r.qlen;
  r.tiles = (r.qlen + tile_tokens - 1) / tile_tokens;
  return r;
}

// Lane l's span, to all lanes.
__device__ __forceinline__ SeqSpan seq_span_of(const SeqSpan& q, int l) {
  SeqSpan r;
  r.q0 = __shfl_sync(0xffffffffu, q.q0, l);
  r.qlen = __shfl_sync(0xffffffffu, q.qlen, l);
  r.k0 = __shfl_sync(0xffffffffu, q.k0, l);
  r.kvlen = __shfl_sync(0xffffffffu, q.kvlen, l);
  r.off = r.kvlen - r.qlen;
  r.tiles = __shfl_sync(0xffffffffu, q.tiles, l);
  return r;
}

// Place of a sequence's first tile among `tokens / tile + n_seq` places: every
// sequence has enough of them behind it for its tiles, whatever the lengths,
// and a place's sequence is found without looking at all of them.
__device__ __forceinline__ int seq_place(const int* cu, int s, int tokens, int tile) {
  return static_cast<int>(static_cast<uint32_t>(min(max(cu[s], 0), tokens)) / static_cast<uint32_t>(tile)) + s;
}

// The last sequence whose first place is at or before `place` (-1: none), by
// the warp, 32 probes at a time.
__device__ __forceinline__ int seq_of_place(const int* cu, int n_seq, int tokens, int tile, int place,
                                            int lane) {
  int lo = 0, hi = n_seq;
  for (;;) {
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + lane * step;
    const uint32_t at = __ballot_sync(0xffffffffu, i < hi && seq_place(cu, min(i, n_seq - 1), tokens, tile) <= place);
    const int k = __popc(at);
    if (k == 0) return -1;
    lo += (k - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) return lo;
  }
}

template <int D, bool FEW>
struct SeqAttnCfg {
  static constexpr int NTHREADS = 384;
  // registers per thread: 2 x 200 + 104 = 3 x 168, what the launch has
  static constexpr int REGS = 168, REGS_SOFT = 200, REGS_REST = 104;
  static constexpr int NSOFT = 256;
  static constexpr int WARP_K = 8, WARP_MMA = 9, WARP_ITEM = 10, WARP_V = 11;
  static constexpr int BK = 128;
  static constexpr int DBOX = D / 64;
  static constexpr int BOX = 128 * 128;  // [128 rows][64 columns], 16 bits
  static constexpr int TILE = BOX * DBOX;
  // rings of K and V blocks; the kernel for few rows has one tile of Q, and
  // what it waits for is memory: more blocks in flight
  static constexpr int NQ = FEW ? 1 : 2;
  static constexpr int NK = D == 128 ? 3 : FEW ? 6 : 4;
  static constexpr int NV = D == 128 ? (FEW ? 3 : 2) : FEW ? 6 : 4;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = NQ * TILE;
  static constexpr int OFF_V = OFF_K + NK * TILE;
  static constexpr int OFF_BAR = OFF_V + NV * TILE;
  static constexpr int B_Q = 0;
  static constexpr int B_TAIL = 1;          // V rows of a last block landed (then cleared behind the end)
  static constexpr int B_KF = 2;            // [NK]
  static constexpr int B_KE = B_KF + NK;    // [NK]
  static constexpr int B_VF = B_KE + NK;    // [NV]
  static constexpr int B_VE = B_VF + NV;    // [NV]
  static constexpr int B_S = B_VE + NV;     // [2] S written
  static constexpr int B_P = B_S + 2;       // [2][2] half of P written, O rescaled (4 warps)
  static constexpr int B_PV = B_P + 4;      // [2] P V of the first half done
  static constexpr int B_DONE = B_PV + 2;   // every product of the item done
  static constexpr int B_OFREE = B_DONE + 1;  // O read (8 warps)
  static constexpr int B_ML = B_OFREE + 1;  // (m, l) of both streams of a one-tile item (8 warps)
  static constexpr int B_X = B_ML + 1;      // few rows: sums in shared memory (8 warps)
  static constexpr int B_DRAIN = B_X + 1;
  static constexpr int NITEM = 2;
  static constexpr int B_IF = B_DRAIN + 1;   // [NITEM] item record written
  static constexpr int B_IE = B_IF + NITEM;  // [NITEM] read (2 loaders, issuer, 8 softmax warps)
  static constexpr int B_NEXT = B_IE + NITEM;  // the item's last K block is on its way
  static constexpr int NBAR = B_NEXT + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  // misc words: [0] tmem base, [1] abort, [3] always 0
  static constexpr int MISC_BYTES = 16;
  static constexpr int OFF_ITEM = OFF_MISC + MISC_BYTES;
  static constexpr int OFF_ML = (OFF_ITEM + NITEM * 48 + 15) / 16 * 16;  // float2 [2][128]
  static constexpr int SMEM_BYTES = OFF_ML + 2 * 128 * 8;
  static constexpr int S_COL = 0;    // stream s at 128 s
  static constexpr int O_COL = 256;  // stream s at 256 + D s
  static constexpr int TMEM_COLS = 512;
  // the reference moves only when a score is more than 2^TAU over where it was set
  static constexpr float TAU = 8.0f;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

// shared list: the cost of an item in units of one stream's key block, with a
// constant for its start and end
constexpr int kSeqItemCost = 4;
constexpr int kSeqMinRange = 10;  // every range inside an item then holds a block's start
constexpr int kSeqMostPiece = 8;  // little work: most blocks of an item per CTA

__device__ __forceinline__ int seq_blocks(const SeqSpan& q, int causal, int tok) {
  const int keys = causal ? min(max(q.off + tok + 1, 0), q.kvlen) : q.kvlen;
  return (keys + 127) >> 7;
}

struct SeqItem {
  int tok0, ntok, nblk, nblk0, unit;
  bool one;  // one tile: both streams share its rows
};

__device__ __forceinline__ SeqItem seq_item(const SeqSpan& q, int causal, int rt, int it_tok, int t) {
  SeqItem it;
  it.tok0 = t * it_tok;
  it.ntok = min(it_tok, q.qlen - it.tok0);
  it.one = it.ntok <= rt;
  it.nblk = seq_blocks(q, causal, it.tok0 + it.ntok - 1);
  it.nblk0 = it.one ? it.nblk : seq_blocks(q, causal, it.tok0 + rt - 1);
  it.unit = it.one ? 1 : 2;
  return it;
}

// Of one KV head of a sequence: its cost, items and key blocks.
struct SeqCost {
  long long cost, items, blocks;
};
__device__ __forceinline__ SeqCost seq_cost(const SeqSpan& q, int causal, int rt, int it_tok) {
  SeqCost c{0, q.tiles, 0};
  for (int t = 0; t < q.tiles; ++t) {
    const SeqItem it = seq_item(q, causal, rt, it_tok, t);
    c.cost += kSeqItemCost + static_cast<long long>(it.nblk) * it.unit;
    c.blocks += it.nblk;
  }
  return c;
}

// Pieces of up to r blocks of an item (an item without blocks is one).
__device__ __forceinline__ int seq_pieces(const SeqItem& it, int r) {
  return it.nblk <= r ? 1 : static_cast<int>(static_cast<uint32_t>(it.nblk + r - 1) / static_cast<uint32_t>(r));
}

// a / b of non-negative numbers; 64-bit division only where it is needed (it
// took a fifth of a short call's kernel).
__device__ __forceinline__ long long seq_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Blocks [b0, b1) of an item that starts at `at` in the list and fall into
// the range [lo, hi): block 0 begins at `at`, block b > 0 behind the constant.
__device__ __forceinline__ int seq_first_block(long long at, const SeqItem& it, long long lo) {
  if (lo <= at) return 0;
  const long long x = lo - at - kSeqItemCost;
  const long long b = x <= 0 ? 1 : (x + it.unit - 1) >> (it.unit - 1);  // unit is 1 or 2
  return static_cast<int>(b < 1 ? 1 : (b > it.nblk ? it.nblk : b));
}

// What the roles need to know of an item; vis + token of the tile: keys a row
// sees (causal), or the sequence's length. seq < 0 ends.
struct SeqRecord {
  static constexpr int kWords = 12;
  static constexpr int kOne = 1, kWhole = 2, kBegins = 4, kFew = 8;
  int hk, qtok, ntok, b0, nb, cnt0, kvlen, k0, vis, seq, mode;
  __device__ __forceinline__ bool one() const { return mode & kOne; }
  __device__ __forceinline__ bool few() const { return mode & kFew; }
  __device__ __forceinline__ int cnt(int st) const {
    return st == 0 ? cnt0 : (one() ? nb >> 1 : nb);
  }
};

template <typename T>
__device__ __forceinline__ uint32_t seq_pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t seq_pack2<__nv_bfloat16>(float lo, float hi) {
  return ptx::pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t seq_pack2<__half>(float lo, float hi) {
  return ptx::pack_f16x2(lo, hi);
}
template <typename T>
__device__ __forceinline__ void seq_unpack2(uint32_t w, float& lo, float& hi);
template <>
__device__ __forceinline__ void seq_unpack2<__nv_bfloat16>(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}
template <>
__device__ __forceinline__ void seq_unpack2<__half>(uint32_t w, float& lo, float& hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  lo = f.x;
  hi = f.y;
}
// kRefBelow: how far under a row's maximum its reference is set, log2. P in fp16
// is then at most 2^(8 + 7), which it holds, and keeps all its bits down to 2^-21
// of the largest P. With the reference at the maximum P would lose bits below
// 2^-14 and be 0 below 2^-25, and a row whose strongest key has a value near 0 is
// made of just those (65536 keys, such a key 18 nats over the rest: error of o
// 0.26, with the 7 less than 1e-4). Moving the reference at 2^4 would leave room
// for 11, and costs 2.5 % (15576 tokens of 32 / 8 heads of 128: 747 -> 766 us).
// bf16 has the exponents of fp32.
template <typename T>
struct SeqType;
template <>
struct SeqType<__nv_bfloat16> {
  static constexpr uint32_t kFormat = 1;
  static constexpr float kRefBelow = 0.0f;
};
template <>
struct SeqType<__half> {
  static constexpr uint32_t kFormat = 0;
  static constexpr float kRefBelow = 7.0f;
};

// Few rows: a lane's sums of both streams over D / 4 columns from `col` on,
// weighted, to shared memory; a weight of 0 takes nothing (the sum may never
// have been written).
template <int D>
__device__ __forceinline__ void seq_few_put(uint32_t o_tm, int col, float* x, float w0, float w1) {
  uint32_t r0[32], r1[32];
  const int skip = col & 31;  // d = 64: half of a load
  ptx::tmem_ld32(o_tm + (col & ~31), r0);
  ptx::tmem_ld32(o_tm + D + (col & ~31), r1);
  ptx::tmem_wait_ld();
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (j < skip || j >= skip + D / 4) continue;
    const float a = w0 == 0.0f ? 0.0f : w0 * __uint_as_float(r0[j]);
    x[(j - skip) * 32] = w1 == 0.0f ? a : fmaf(w1, __uint_as_float(r1[j]), a);
  }
}

// Adds up the four quarters' sums of a row over D / 16 columns; to `part`
// (fp32) if there is one, else to `o`.
template <int D, typename T>
__device__ __forceinline__ void seq_few_take(const float* x, T* o, float* part) {
  constexpr int Q = D / 4 * 32;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float* y = x + (4 * c + j) * 32;
      v[j] = (y[0] + y[Q]) + (y[2 * Q] + y[3 * Q]);
    }
    if (part) *reinterpret_cast<float4*>(part + 4 * c) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2*>(o + 4 * c) = make_uint2(seq_pack2<T>(v[0], v[1]), seq_pack2<T>(v[2], v[3]));
  }
}

template <int N>
struct SeqInt {
  static constexpr int value = N;
};

template <int D, typename T, bool FEW>
__global__ void __launch_bounds__(384, 1)
    blasst_seq_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                           const __grid_constant__ CUtensorMap tmQFew,
                           const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const SeqAttnParams p) {
  using C = SeqAttnCfg<D, FEW>;
  constexpr uint32_t IDESC_S = ptx::idesc_f32acc(SeqType<T>::kFormat, 128, 128, false);
  constexpr uint32_t IDESC_PV = ptx::idesc_f32acc(SeqType<T>::kFormat, 128, D, true);
  constexpr float BELOW = SeqType<T>::kRefBelow;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  const uint32_t sb = ptx::smem_u32(smem);
  volatile int* misc = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  volatile int* abort_flag = misc + 1;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8 * i; };
  if ((sb & 1023u) != 0u) {  // uniform; the tiles need 1 KB alignment
    if (threadIdx.x == 0) seq_record_error(p.err, BLASST_EUNSUPPORTED);
    return;
  }

  volatile int* items = reinterpret_cast<volatile int*>(smem + C::OFF_ITEM);

  // ---- set-up --------------------------------------------------------------
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NITEM; ++i) {
      ptx::mbar_init(bar(C::B_IF + i), 1);
      ptx::mbar_init(bar(C::B_IE + i), 11);
    }
    ptx::mbar_init(bar(C::B_Q), 1);
    ptx::mbar_init(bar(C::B_TAIL), 1);
    for (int i = 0; i < 2 * (C::NK + C::NV); ++i) ptx::mbar_init(bar(C::B_KF + i), 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(C::B_S + i), 1);
      ptx::mbar_init(bar(C::B_P + 2 * i), 4);
      ptx::mbar_init(bar(C::B_P + 2 * i + 1), 4);
      ptx::mbar_init(bar(C::B_PV + i), 1);
    }
    ptx::mbar_init(bar(C::B_DONE), 1);
    ptx::mbar_init(bar(C::B_OFREE), 8);
    ptx::mbar_init(bar(C::B_ML), 8);
    ptx::mbar_init(bar(C::B_X), 8);
    ptx::mbar_init(bar(C::B_DRAIN), 1);
    ptx::mbar_init(bar(C::B_NEXT), 1);
    for (int i = 1; i < 4; ++i) misc[i] = 0;
    ptx::fence_mbar_init();
  }
  if (warp == C::WARP_MMA) {
    ptx::tmem_alloc(ptx::smem_u32(const_cast<int*>(misc)), C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  auto span = [&](int s) -> SeqSpan {
    if (s < 0 || s >= p.n_seq) return SeqSpan{};
    const int kv_cap = static_cast<int>(
        min(static_cast<long long>(p.table_width) * p.page_size, 0x7fffff00ll));
    return seq_span(p.cu_q, p.cu_k, p.kv_lens, kv_cap, p.Tq, p.Tk, p.it_tok, s, p.err);
  };
  // whole item i, the last tiles of a head first: its sequence (-1: none) and tile
  auto find = [&](int i, SeqSpan& q, int& t) -> int {
    const int place = p.n_tiles - 1 - i % p.n_tiles;
    const int s = seq_of_place(p.cu_q, p.n_seq, p.Tq, p.it_tok, place, lane);
    if (s < 0) return -1;
    q = span(s);
    t = place - seq_place(p.cu_q, s, p.Tq, p.it_tok);
    return t < q.tiles ? s : -1;
  };
  // beside the set-up: the CTA's first whole item, or the lane's sequence of the
  // shared list
  SeqSpan first_q{};
  int first_s = -1, first_t = 0;
  if (warp == C::WARP_ITEM) {
    if (p.n_tiles != 0) first_s = find(static_cast<int>(blockIdx.x), first_q, first_t);
    else first_q = span(lane);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);

  // Item n of the CTA as a role reads it: all lanes get the record, the role
  // hands the slot back at once (`releases`: one arrival of this warp).
  auto next_item = [&](int n, SeqRecord& r) -> bool {
    const int slot = n % C::NITEM;
    if (!ptx::mbar_wait(bar(C::B_IF + slot), (n / C::NITEM) & 1, abort_flag, p.timeout_ns))
      return false;
    const volatile int* w = items + slot * SeqRecord::kWords;
    r.hk = w[0];
    r.qtok = w[1];
    r.ntok = w[2];
    r.b0 = w[3];
    r.nb = w[4];
    r.cnt0 = w[5];
    r.kvlen = w[6];
    r.k0 = w[7];
    r.vis = w[8];
    r.seq = w[9];
    r.mode = w[10];
    return true;
  };
  auto item_read = [&](int n) { ptx::mbar_arrive(bar(C::B_IE + n % C::NITEM)); };
  auto fail = [&]() {
    *abort_flag = 1;
    seq_record_error(p.err, BLASST_ETIMEOUT);
  };

  ptx::grid_launch_dependents();  // the join's blocks may come up meanwhile
  if (warp >= 8) {
   ptx::reg_give<C::REGS_REST>();
   if (warp == C::WARP_ITEM) {
    // ======================= the CTA's items ================================
    int n = 0;
    auto put = [&](int s, const SeqSpan& q, int h, const SeqItem& it, int b0, int b1) -> bool {
      const int slot = n % C::NITEM;
      bool ok = true;
      if (n >= C::NITEM)
        ok = ptx::mbar_wait(bar(C::B_IE + slot), ((n / C::NITEM) - 1) & 1, abort_flag, p.timeout_ns);
      ok = __all_sync(0xffffffffu, ok) != 0;
      if (!ok) return false;
      if (lane == 0) {
        volatile int* w = items + slot * SeqRecord::kWords;
        const bool whole = b0 == 0 && b1 == it.nblk;
        w[0] = h;
        w[1] = q.q0 + it.tok0;
        w[2] = s < 0 ? 0 : it.ntok;
        w[3] = b0;
        w[4] = b1 - b0;
        w[5] = it.one ? (b1 - b0 + 1) >> 1 : max(min(b1, it.nblk0) - b0, 0);
        w[6] = q.kvlen;
        w[7] = q.k0;
        w[8] = p.causal ? q.off + it.tok0 + 1 : q.kvlen;
        w[9] = s;
        w[10] = (it.one ? SeqRecord::kOne : 0) | (whole ? SeqRecord::kWhole : 0) |
                (FEW && it.one && it.ntok <= p.rt_few ? SeqRecord::kFew : 0) |
                (b0 == 0 ? SeqRecord::kBegins : 0);
        ptx::mbar_arrive(bar(C::B_IF + slot));
      }
      ++n;
      return true;
    };
    // after a wait gave up, calls before blasst_check do nothing
    const bool live = !(p.err && *reinterpret_cast<volatile int*>(p.err) == BLASST_ETIMEOUT);
    bool ok = true;
    if (p.n_tiles != 0) {
      // ---- whole items -----------------------------------------------------
      // One, or the CTA's first and then one after the other from the list of
      // all, each taken when the one before has its last K block on its way
      // (sooner would leave the list's end less even, later K's ring empty).
      const int count = p.n_tiles * p.Hkv;
      int i = static_cast<int>(blockIdx.x);
      SeqSpan q = first_q;
      int s = first_s, t = first_t;
      while (live && i < count) {
        if (s >= 0) {
          const SeqItem it = seq_item(q, p.causal, p.rt, p.it_tok, t);
          ok = put(s, q, i / p.n_tiles, it, 0, it.nblk);
          if (ok && p.next) ok = ptx::mbar_wait(bar(C::B_NEXT), (n - 1) & 1, abort_flag, p.timeout_ns);
          ok = __all_sync(0xffffffffu, ok) != 0;
          if (!ok) break;
        }
        if (!p.next) break;
        if (lane == 0) i = static_cast<int>(gridDim.x) + atomicAdd(p.next, 1);
        i = __shfl_sync(0xffffffffu, i, 0);
        if (i < count) s = find(i, q, t);
      }
    } else {
      // ---- this CTA's range of the shared list -----------------------------
      // no item cut at the range's end, until one is found
      if (lane == 0) p.part_desc[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
      // the sequences' spans are read 32 U at a time, U per lane; up to that
      // many are read once (one per lane while that is enough: four took 6 us
      // more of a call with three sequences)
      auto my_part = [&](auto per_lane) {
        constexpr int U = decltype(per_lane)::value, CHUNK = 32 * U;
        int chunk = U == 1 ? 0 : -1;
        SeqSpan mine[U];
        mine[0] = first_q;
        auto load_chunk = [&](int s0) {
          if (s0 == chunk) return;
#pragma unroll
          for (int u = 0; u < U; ++u) mine[u] = span(s0 + lane * U + u);
          chunk = s0;
        };
        auto span_of = [&](int s) -> SeqSpan {
          load_chunk(s & ~(CHUNK - 1));
          SeqSpan r = mine[0];
#pragma unroll
          for (int u = 1; u < U; ++u)
            if ((s & (U - 1)) == u) r = mine[u];
          return seq_span_of(r, (s & (CHUNK - 1)) / U);
        };
        long long total = 0, items = 0, blocks = 0, own = 0;
        auto add_up = [&](long long c) -> long long {
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) c += __shfl_xor_sync(0xffffffffu, c, d);
          return c;
        };
        auto lane_cost = [&]() -> long long {
          long long c = 0;
#pragma unroll
          for (int u = 0; u < U; ++u) c += seq_cost(mine[u], p.causal, p.rt, p.it_tok).cost;
          return c * p.Hkv;
        };
        for (int s0 = 0; s0 < p.n_seq; s0 += CHUNK) {
          load_chunk(s0);
          SeqCost c{0, 0, 0};
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const SeqCost one = seq_cost(mine[u], p.causal, p.rt, p.it_tok);
            c.cost += one.cost;
            c.items += one.items;
            c.blocks += one.blocks;
          }
          own = c.cost * p.Hkv;
          total += add_up(own);
          items += add_up(c.items) * p.Hkv;
          blocks += add_up(c.blocks) * p.Hkv;
        }
        // Little work (an eighth of a CTA's worth of items to spare, few blocks
        // each): every CTA one piece of one item, so that none has to start
        // another item behind its first.
        const long long spare = static_cast<long long>(gridDim.x) - items;
        const long long piece = spare > 0 ? max(2ll, seq_div(blocks + spare - 1, spare)) : 0;
        const bool little = 8 * spare >= gridDim.x && piece <= kSeqMostPiece;
        if (little) {
          const int r = static_cast<int>(piece);
          long long at = 0;
          auto pieces_of = [&](const SeqSpan& q) -> long long {
            long long n_pieces = 0;
            for (int t = 0; t < q.tiles; ++t)
              n_pieces += seq_pieces(seq_item(q, p.causal, p.rt, p.it_tok, t), r);
            return n_pieces;
          };
          for (int s0 = 0; s0 < p.n_seq && live; s0 += CHUNK) {
            load_chunk(s0);
            long long np = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) np += pieces_of(mine[u]) * p.Hkv;
            long long upto = np;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
              const long long v = __shfl_up_sync(0xffffffffu, upto, d);
              if (lane >= d) upto += v;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, blockIdx.x < at + upto);
            if (hit) {
              const int l = __ffs(hit) - 1;
              at += __shfl_sync(0xffffffffu, upto - np, l);
              int s = s0 + l * U;  // one of the lane's sequences
              SeqSpan q = span_of(s);
              long long per = pieces_of(q);
              while (blockIdx.x >= at + per * p.Hkv) {
                at += per * p.Hkv;
                q = span_of(++s);
                per = pieces_of(q);
              }
              int left = static_cast<int>(blockIdx.x - at);
              const int h = left / static_cast<int>(per);
              left -= h * static_cast<int>(per);
              SeqItem it = seq_item(q, p.causal, p.rt, p.it_tok, 0);
              int n_pieces = seq_pieces(it, r);
              for (int t = 1; left >= n_pieces; ++t) {
                left -= n_pieces;
                it = seq_item(q, p.causal, p.rt, p.it_tok, t);
                n_pieces = seq_pieces(it, r);
              }
              if (lane == 0 && left == 0 && n_pieces > 1) {
                p.part_desc[2 * blockIdx.x] = make_int4(q.q0 + it.tok0, it.ntok, h, it.one ? 1 : 0);
                p.part_desc[2 * blockIdx.x + 1] = make_int4(blockIdx.x + n_pieces - 1, 0, 0, 0);
              }
              ok = put(s, q, h, it, left * r, min(left * r + r, it.nblk));
              break;
            }
            at += __shfl_sync(0xffffffffu, upto, 31);
          }
        }
        const long long share = seq_div(total + gridDim.x - 1, gridDim.x);
        const long long range = share < kSeqMinRange ? kSeqMinRange : share;
        const long long lo = range * blockIdx.x;
        const long long hi = lo + range < total ? lo + range : total;
        long long at = 0;  // the list's place of what is looked at
        int s = 0, h = 0, t = 0;
        bool found = false;
        for (int s0 = 0; s0 < p.n_seq && !found && !little && live && lo < total; s0 += CHUNK) {
          if (s0 != chunk) {
            load_chunk(s0);
            own = lane_cost();
          }
          long long upto = own;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += v;
          }
          const uint32_t hit = __ballot_sync(0xffffffffu, lo < at + upto);
          if (hit) {
            const int l = __ffs(hit) - 1;
            at += __shfl_sync(0xffffffffu, upto - own, l);
            s = s0 + l * U;  // one of the lane's sequences
            long long per = seq_cost(span_of(s), p.causal, p.rt, p.it_tok).cost;
            while (lo >= at + per * p.Hkv) {
              at += per * p.Hkv;
              per = seq_cost(span_of(++s), p.causal, p.rt, p.it_tok).cost;
            }
            h = static_cast<int>(seq_div(lo - at, per));
            at += h * per;
            found = true;
          } else {
            at += __shfl_sync(0xffffffffu, upto, 31);
          }
        }
        if (found) {
          SeqSpan q = span_of(s);
          while (at < hi && ok) {
            const SeqItem it = seq_item(q, p.causal, p.rt, p.it_tok, t);
            const long long end = at + kSeqItemCost + static_cast<long long>(it.nblk) * it.unit;
            if (end > lo) {
              const int b0 = it.nblk ? seq_first_block(at, it, lo) : 0;
              const int b1 = it.nblk ? seq_first_block(at, it, hi) : 0;
              // (an item that begins before the range and has no block that
              // starts in it is the range before's)
              if (at >= lo || b0 < b1) {
                if (lane == 0 && b0 == 0 && b1 < it.nblk) {
                  // it goes on in the ranges behind this one: what the join needs
                  p.part_desc[2 * blockIdx.x] =
                      make_int4(q.q0 + it.tok0, it.ntok, h, it.one ? 1 : 0);
                  p.part_desc[2 * blockIdx.x + 1] =
                      make_int4(static_cast<int>(seq_div(end - it.unit, range)), 0, 0, 0);
                }
                ok = put(s, q, h, it, b0, b1);
              }
            }
            at = end;
            if (++t == q.tiles) {
              t = 0;
              if (++h == p.Hkv) {
                h = 0;
                do {
                  if (++s >= p.n_seq) break;
                  q = span_of(s);
                } while (q.tiles == 0);
                if (s >= p.n_seq) break;
              }
            }
          }
        }
      };
      if (p.n_seq <= 32) my_part(SeqInt<1>{});
      else my_part(SeqInt<4>{});
    }
    if (ok) {
      SeqSpan q{};
      SeqItem it{};
      ok = put(-1, q, 0, it, 0, 0);  // the end
    }
    if (!ok && lane == 0) fail();
  } else if (warp == C::WARP_K || warp == C::WARP_V) {
    // ======================= TMA producers =================================
    // One warp for K (and Q), one for V. Their own time per block counts: with
    // one warp for both, a table entry read per block and divisions in the
    // loop, a step of single tokens was bound by it.
    const bool is_v = warp == C::WARP_V;
    const CUtensorMap* tm = is_v ? &tmV : &tmK;
    const uint32_t depth = is_v ? C::NV : C::NK;
    const int b_full = is_v ? C::B_VF : C::B_KF, b_empty = is_v ? C::B_VE : C::B_KE;
    const int ring_off = is_v ? C::OFF_V : C::OFF_K;
    if (lane == 0) {
      ptx::prefetch_tmap(tm);
      if (!is_v) ptx::prefetch_tmap(FEW ? &tmQFew : &tmQ);
    }
    const int chunk = 1 << p.chunk_log2;
    const int nch_log2 = 7 - p.chunk_log2, nch = 1 << nch_log2;
    const int q_box_rows = p.g * p.rt;
    // Places in the cache (page, row in it) are looked up a group of 32 chunks
    // (one per lane) at a time, one group ahead of their use.
    const int group_log2 = 5 - nch_log2;  // blocks of a group
    int2 at_now = make_int2(0, 0), at_next = at_now;
    int group = -1;
    uint32_t ring = 0;            // loads issued
    uint32_t slot = 0, turn = 0;  // of the ring; turn: parity of the slot's phase
    uint32_t tails = 0;           // cleared last blocks
    bool ok = true;
    bool last_tail = false;
    int q_loads = 0;
    bool few_before = false;
    SeqRecord it;
    auto load_q = [&](int n) -> bool {
      // once the item before has finished with it (the first K blocks do not
      // wait for that); few rows leave their sums in Q's place
      if (n > 0 && !ptx::mbar_wait(bar(C::B_DONE), (n - 1) & 1, abort_flag, p.timeout_ns)) return false;
      // (only behind the wait above is the phase before known to be over)
      if (FEW && few_before &&
          !ptx::mbar_wait(bar(C::B_OFREE), (n - 1) & 1, abort_flag, p.timeout_ns))
        return false;
      const bool few = FEW && it.few();
      const int parts = few ? 4 : it.one() ? 1 : 2;
      ptx::mbar_arrive_expect_tx(bar(C::B_Q),
                                 parts * C::DBOX * (few ? p.g * p.rt_few : q_box_rows) * 128);
      for (int i = 0; i < parts; ++i)
#pragma unroll
        for (int x = 0; x < C::DBOX; ++x) {
          if (few)
            ptx::tma_load_4d(sb + C::OFF_Q + x * C::BOX + i * 32 * 128, &tmQFew, x * 64, 0, it.qtok,
                             it.hk, bar(C::B_Q));
          else
            ptx::tma_load_4d(sb + C::OFF_Q + i * C::TILE + x * C::BOX, &tmQ, x * 64, 0,
                             it.qtok + i * p.rt, it.hk, bar(C::B_Q));
        }
      q_loads = n + 1;
      return true;
    };
    for (int n = 0; ok; ++n) {
      ok = __all_sync(0xffffffffu, next_item(n, it)) != 0;
      if (!ok) break;
      if (lane == 0) item_read(n);
      if (it.seq < 0) break;
      const int nb = it.nb;
      auto read_group = [&](int gr) -> int2 {
        const long long key = (static_cast<long long>(gr) * 32 + lane) << p.chunk_log2;
        if (key >= it.kvlen) return make_int2(p.n_pages, 0);
        const int k = static_cast<int>(key);
        return make_int2(p.table[static_cast<long long>(it.seq) * p.table_stride + k / p.page_size],
                         k % p.page_size);
      };
      if (p.table) {
        group = it.b0 >> group_log2;
        at_now = read_group(group);
        at_next = read_group(group + 1);
      }
      const int q_at = n == 0 ? 0 : min(nb, 2);
      for (int b = 0; b <= nb && ok; ++b) {
        if (!is_v && b == q_at) {
          if (lane == 0) ok = load_q(n);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          few_before = it.few();
        }
        if (b == nb || !ok) {
          if (!is_v && ok && lane == 0) ptx::mbar_arrive(bar(C::B_NEXT));
          break;
        }
        const int key0 = (it.b0 + b) * C::BK;
        const int valid = min(C::BK, it.kvlen - key0);
        // this lane's piece of the block
        int row = it.k0 + key0, page = 0;
        const bool mine = lane < nch && (lane << p.chunk_log2) < valid;
        if (p.table) {
          const int block = it.b0 + b;
          if ((block >> group_log2) > group) {
            ++group;
            at_now = at_next;
            at_next = read_group(group + 1);
          }
          const int from = ((block & ((1 << group_log2) - 1)) << nch_log2) + (lane & (nch - 1));
          page = __shfl_sync(0xffffffffu, at_now.x, from);
          row = __shfl_sync(0xffffffffu, at_now.y, from);
          if (mine && static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) {
            seq_record_error(p.err, BLASST_EINDEX);
            page = p.n_pages;  // outside the map: zeros
          }
        }
        const uint32_t full = bar(b_full + slot);
        const bool tail = is_v && valid < C::BK;
        const uint32_t fb = tail ? bar(C::B_TAIL) : full;
        if (lane == 0) {
          if (ring >= depth)
            ok = ptx::mbar_wait(bar(b_empty + slot), turn ^ 1u, abort_flag, p.timeout_ns);
          if (ok)
            ptx::mbar_arrive_expect_tx(fb, ((valid + chunk - 1) >> p.chunk_log2 << p.chunk_log2) *
                                               (128 * C::DBOX));
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        const int dst = ring_off + static_cast<int>(slot) * C::TILE;
        if (mine) {
#pragma unroll
          for (int x = 0; x < C::DBOX; ++x)
            ptx::tma_load_4d(sb + dst + x * C::BOX + (lane << p.chunk_log2) * 128, tm, x * 64, row,
                             it.hk, page, fb);
        }
        ++ring;
        last_tail = tail;
        if (tail) {
          // Rows behind the sequence's end (a neighbour's, a page's leftovers,
          // an earlier block's) may hold anything, and 0 x NaN is NaN: clear
          // them. K needs no clearing, its scores are replaced.
          ok = ptx::mbar_wait(bar(C::B_TAIL), tails & 1, abort_flag, p.timeout_ns);
          ok = __all_sync(0xffffffffu, ok) != 0;
          ++tails;
          if (!ok) break;
          for (int i = valid * 8 + lane; i < C::BK * 8; i += 32)
#pragma unroll
            for (int x = 0; x < C::DBOX; ++x)
              *reinterpret_cast<uint4*>(smem + dst + x * C::BOX + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(full);
          last_tail = false;
        }
        if (++slot == depth) {
          slot = 0;
          turn ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      fail();
      // copies in flight land before the CTA exits (1 ms each is ample)
      const uint64_t drain_ns = p.timeout_ns < 1000000ull ? p.timeout_ns : 1000000ull;
      for (uint32_t k = ring < depth ? 0 : ring - depth; k < ring; ++k)
        if (!(last_tail && k + 1 == ring))
          ptx::mbar_wait(bar(b_full + k % depth), (k / depth) & 1, &misc[3], drain_ns);
      if (last_tail) ptx::mbar_wait(bar(C::B_TAIL), (tails - 1) & 1, &misc[3], drain_ns);
      if (q_loads > 0) ptx::mbar_wait(bar(C::B_Q), (q_loads - 1) & 1, &misc[3], drain_ns);
    }
  } else if (warp == C::WARP_MMA) {
    // ======================= tcgen05 issuer ================================
    // What this thread does between two products is time the tensor core does
    // not work: ring places are kept as counters, descriptors are ready before
    // the waits, a block that both streams use is waited for once, and the lane
    // is an elected one, which the compiler knows to be alone (2 % over lane 0).
    if (ptx::elect_one()) {
      bool ok = true;
      const uint64_t q_desc = ptx::sw128_desc(sb + C::OFF_Q, 16, 1024);
      const uint64_t k_desc = ptx::sw128_desc(sb + C::OFF_K, 16, 1024);
      const uint64_t v_desc = ptx::sw128_desc(sb + C::OFF_V, C::BOX, 1024);
      constexpr uint64_t TS = C::TILE >> 4;
      uint32_t k_slot = 0, k_turn = 0, v_slot = 0, v_turn = 0;  // newest blocks, phase parity
      uint64_t kd = k_desc, vd = v_desc;                        // of those slots
      uint32_t phase[2] = {0, 0};                               // of P, per stream
      SeqRecord it;
      auto wait = [&](int b, uint32_t parity) -> bool {
        return ptx::mbar_wait(bar(b), parity, abort_flag, p.timeout_ns);
      };
      for (int n = 0; ok; ++n) {
        ok = next_item(n, it);
        if (!ok) break;
        item_read(n);
        if (it.seq < 0) break;
        const bool one = it.one();
        const int cnt0 = it.cnt(0), cnt1 = it.cnt(1);
        ok = wait(C::B_Q, n & 1);
        if (!ok) break;
        // S of stream st; `first`: of the streams that use the block, `last` too
        auto issue_s = [&](auto stream, bool first, bool last) -> bool {
          constexpr int st = decltype(stream)::value;
          const uint64_t qd = q_desc + (st == 1 && !one ? TS : 0);
          if (first && !wait(C::B_KF + k_slot, k_turn)) return false;
          ptx::tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t o = static_cast<uint64_t>(((kk >> 2) * C::BOX + (kk & 3) * 32) >> 4);
            ptx::mma_ss(tmem + C::S_COL + st * 128, qd + o, kd + o, IDESC_S, kk > 0 ? 1u : 0u);
          }
          ptx::mma_commit(bar(C::B_S + st));
          if (last) {
            ptx::mma_commit(bar(C::B_KE + k_slot));
            kd += TS;
            if (++k_slot == C::NK) {
              k_slot = 0;
              k_turn ^= 1u;
              kd = k_desc;
            }
          }
          return true;
        };
        auto issue_pv = [&](auto stream, int i, bool first, bool last) -> bool {
          constexpr int st = decltype(stream)::value;
          const uint32_t o_tm = tmem + C::O_COL + st * D;
          const uint32_t p_tm = tmem + C::S_COL + st * 128;
          if (first && !wait(C::B_VF + v_slot, v_turn)) return false;
          // the first half of the keys as soon as its P is there
          if (!wait(C::B_P + 2 * st, phase[st])) return false;
          ptx::tc_fence_after();
          ptx::mma_ts(o_tm, p_tm, vd, IDESC_PV, i > 0 ? 1u : 0u);
#pragma unroll
          for (int kk = 1; kk < C::BK / 32; ++kk)
            ptx::mma_ts(o_tm, p_tm + kk * 8, vd + static_cast<uint64_t>(kk * (2048 >> 4)), IDESC_PV, 1u);
          ptx::mma_commit(bar(C::B_PV + st));
          if (!wait(C::B_P + 2 * st + 1, phase[st])) return false;
          ptx::tc_fence_after();
#pragma unroll
          for (int kk = C::BK / 32; kk < C::BK / 16; ++kk)
            ptx::mma_ts(o_tm, p_tm + kk * 8, vd + static_cast<uint64_t>(kk * (2048 >> 4)), IDESC_PV, 1u);
          phase[st] ^= 1u;
          if (last) {
            ptx::mma_commit(bar(C::B_VE + v_slot));
            vd += TS;
            if (++v_slot == C::NV) {
              v_slot = 0;
              v_turn ^= 1u;
              vd = v_desc;
            }
          }
          return true;
        };
        // two tiles: stream 1 sees every block, stream 0 the first cnt0 of them
        const SeqInt<0> s0;
        const SeqInt<1> s1;
        if (cnt0 > 0) ok = issue_s(s0, true, one);
        if (ok && cnt1 > 0) ok = issue_s(s1, one || cnt0 == 0, true);
        // O is free once the item before has been read out
        if (ok && n > 0) ok = wait(C::B_OFREE, (n - 1) & 1);
        const int most = max(cnt0, cnt1);
        for (int i = 0; i < most && ok; ++i) {
          if (i < cnt0) {
            ok = issue_pv(s0, i, true, one);
            if (ok && i + 1 < cnt0) ok = issue_s(s0, true, one);
          }
          if (ok && i < cnt1) {
            ok = issue_pv(s1, i, one || i >= cnt0, true);
            if (ok && i + 1 < cnt1) ok = issue_s(s1, one || i + 1 >= cnt0, true);
          }
        }
        ptx::mma_commit(bar(C::B_DONE));
      }
      if (!ok) fail();
      // every product has completed before TMEM is freed
      ptx::mma_commit(bar(C::B_DRAIN));
      ptx::mbar_wait(bar(C::B_DRAIN), 0, &misc[3], p.timeout_ns);
    }
   }
  } else {
    ptx::reg_take<C::REGS_SOFT>();
    // ======================= softmax =======================================
    const int st = warp >> 2;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;  // row of the tile, TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + C::S_COL + st * 128;
    const uint32_t o_tm = tmem + lane_base + C::O_COL + st * D;
    const float sl2 = p.scale_log2;
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    uint32_t steps = 0;  // blocks done (S phases)
    uint32_t ones = 0;   // one-tile items done
    bool ok = true;
    auto lane0_wait = [&](uint32_t b, uint32_t parity) -> bool {
      bool r = true;
      if (lane == 0) r = ptx::mbar_wait(b, parity, abort_flag, p.timeout_ns);
      return __shfl_sync(0xffffffffu, r ? 1 : 0, 0) != 0;
    };
    auto scale_o = [&](float alpha) {
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t r[32];
        ptx::tmem_ld32(o_tm + 32 * c, r);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * alpha);
        ptx::tmem_st32(o_tm + 32 * c, r);
      }
    };
    uint32_t meets = 0;  // B_X phases
    SeqRecord it;
    for (int n = 0; ok; ++n) {
      ok = __all_sync(0xffffffffu, next_item(n, it)) != 0;
      if (!ok) break;
      if (lane == 0) item_read(n);
      if (it.seq < 0) break;
      const bool one = it.one(), few = FEW && it.few();
      const int cnt = it.cnt(st);
      const int first_tok = one ? 0 : st * p.rt;
      const int row_tok = (few ? lane : row) / p.g, row_head = (few ? lane : row) % p.g;
      const int tok = first_tok + row_tok;  // of the item
      const bool exists = row_tok < (few ? p.rt_few : p.rt) && tok < it.ntok;
      const bool active = __any_sync(0xffffffffu, exists) != 0;
      // keys below `limit` are visible; the tile's first token sees the fewest
      const int limit = p.causal ? min(it.vis + tok, it.kvlen) : it.kvlen;
      const int least = p.causal ? min(it.vis + first_tok, it.kvlen) : it.kvlen;
      float mref = -INFINITY, l = 0.0f;
      if (few) {
        for (int i = 0; i < cnt; ++i) {
          const int col0 = (it.b0 + (one ? 2 * i + st : i)) * C::BK;
          ok = lane0_wait(bar(C::B_S + st), steps & 1);
          ++steps;
          if (!ok) break;
          ptx::tc_fence_after();
          // this quarter's 32 keys of the block
          uint32_t sv[32];
          ptx::tmem_ld32(s_tm + 32 * quad, sv);
          ptx::tmem_wait_ld();
          const int vis = limit - col0 - 32 * quad;
          if (col0 + C::BK > least) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c >= vis) sv[c] = __float_as_uint(-INFINITY);
          }
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            mx[0] = ptx::fmax3(mx[0], __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
            mx[1] = ptx::fmax3(mx[1], __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
          }
          const float mb = fmaxf(mx[0], mx[1]) * sl2;
          const bool need = mb > mref + (C::TAU + BELOW);
          if (__any_sync(0xffffffffu, need)) {
            const float mnew = need ? mb - BELOW : mref;
            const float alpha = need ? ptx::ex2(mref - mnew) : 1.0f;
            mref = mnew;
            l *= alpha;
            if (i > 0) scale_o(alpha);
          }
          const float neg = mref == -INFINITY ? 0.0f : -mref;
          float rs[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t pk[16], zero[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float x0, x1;
            ptx::fma2(x0, x1, __uint_as_float(sv[j]), __uint_as_float(sv[j + 1]), sl2, sl2, neg, neg);
            const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
            const int a = j & 2;
            ptx::add2(rs[a], rs[a + 1], rs[a], rs[a + 1], p0, p1);
            pk[j / 2] = seq_pack2<T>(p0, p1);
            zero[j / 2] = 0u;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q == quad) ptx::tmem_st16(s_tm + 16 * q, pk);
            else ptx::tmem_st16(s_tm + 16 * q, zero);
          }
          l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(bar(C::B_P + 2 * st));
            ptx::mbar_arrive(bar(C::B_P + 2 * st + 1));
          }
        }
      } else {
        for (int i = 0; i < cnt; ++i) {
          const int col0 = (it.b0 + (one ? 2 * i + st : i)) * C::BK;
          ok = lane0_wait(bar(C::B_S + st), steps & 1);
          ++steps;
          if (!ok) break;
          ptx::tc_fence_after();
          if (!active) {
            if (lane == 0) {
              ptx::mbar_arrive(bar(C::B_P + 2 * st));
              ptx::mbar_arrive(bar(C::B_P + 2 * st + 1));
            }
            continue;
          }
          // Two halves of 64 keys. Each takes its exponentials by the reference
          // so far, with the maximum found beside them, and takes them again in
          // the rare case that the reference has to move; its P is handed on at
          // once, so that P V of the first half runs under the second's
          // exponentials.
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t sv[64], pk[32];
            ptx::tmem_ld32p(s_tm + 64 * h, sv);
            ptx::tmem_ld32p(s_tm + 64 * h + 32, sv + 32);
            ptx::tmem_wait_ld();
            if (col0 + C::BK > least) {
              const int vis = limit - col0 - 64 * h;
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (c >= vis) sv[c] = __float_as_uint(-INFINITY);
            }
            float sum;
            for (;;) {
              const float neg = mref == -INFINITY ? 0.0f : -mref;
              float rs[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
              float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int j = 0; j < 64; j += 2) {
                const float s0 = __uint_as_float(sv[j]), s1 = __uint_as_float(sv[j + 1]);
                float x0, x1;
                ptx::fma2(x0, x1, s0, s1, sl2, sl2, neg, neg);
                const int m = (j >> 1) & 3, a = j & 6;
                mx[m] = ptx::fmax3(mx[m], s0, s1);
                const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
                ptx::add2(rs[a], rs[a + 1], rs[a], rs[a + 1], p0, p1);
                pk[j / 2] = seq_pack2<T>(p0, p1);
              }
              sum = ((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7]));
              const float mb = fmaxf(ptx::fmax3(mx[0], mx[1], mx[2]), mx[3]) * sl2;
              const bool need = mb > mref + (C::TAU + BELOW);  // the first keys of a row always move it
              if (!__any_sync(0xffffffffu, need)) break;
              const float mnew = need ? mb - BELOW : mref;
              const float alpha = need ? ptx::ex2(mref - mnew) : 1.0f;  // 0 from -inf
              mref = mnew;
              l *= alpha;
              // O is quiet: S of this block was issued behind the P V of the one
              // before, and the first half's is waited for
              if (h == 1) {
                ok = lane0_wait(bar(C::B_PV + st), (steps - 1) & 1);
                if (!ok) break;
                ptx::tc_fence_after();
              }
              if (h == 1 || i > 0) scale_o(alpha);
            }
            if (!ok) break;
            ptx::tmem_st32(s_tm + 32 * h, pk);
            l += sum;
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(C::B_P + 2 * st + h));
          }
          if (!ok) break;
        }
      }

      // ---- the item's end ---------------------------------------------------
      if (!ok) break;
      float w0 = 1.0f, w1 = 0.0f;
      if (one) {
        // (the item before has been read out by all warps: ml may be written)
        if (n > 0) ok = lane0_wait(bar(C::B_OFREE), (n - 1) & 1);
        ml[st * 128 + row] = make_float2(mref, l);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_ML));
        ok = lane0_wait(bar(C::B_ML), ones & 1) && ok;
        ++ones;
        if (!ok) break;
        const float2 a = ml[row], c = ml[128 + row];
        mref = fmaxf(a.x, c.x);
        if (few) {
          for (int q = 0; q < 4; ++q)
            mref = ptx::fmax3(mref, ml[32 * q + lane].x, ml[128 + 32 * q + lane].x);
        }
        w0 = a.x == -INFINITY ? 0.0f : ptx::ex2(a.x - mref);
        w1 = c.x == -INFINITY ? 0.0f : ptx::ex2(c.x - mref);
        l = a.y * w0 + c.y * w1;
        if (few) {
          l = 0.0f;
          for (int q = 0; q < 8; ++q) {
            const float2 b = ml[32 * q + lane];
            if (b.x != -INFINITY) l = fmaf(b.y, ptx::ex2(b.x - mref), l);
          }
        }
      }
      ok = lane0_wait(bar(C::B_DONE), n & 1);
      ok = ok && *abort_flag == 0;
      ok = __all_sync(0xffffffffu, ok) != 0;
      if (!ok) break;
      ptx::tc_fence_after();
      // 0 where the row saw no key; NaN (from NaN inputs) stays
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const float lse2 = l == 0.0f ? -INFINITY : mref + log2f(l);
      const bool whole = it.mode & SeqRecord::kWhole;
      const long long tok_row = static_cast<long long>(it.qtok + tok) * p.Hq + it.hk * p.g + row_head;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (it.mode & SeqRecord::kBegins ? 1 : 0);
      const int prow = few ? lane : (one ? 0 : st * 128) + row;
      // one tile: each warpgroup takes half of the columns of both sums
      const int c_lo = one ? st * (D / 64) : 0;
      const int c_hi = one ? c_lo + D / 64 : D / 32;
      const bool second = one && it.nb > 1;
      if (few) {
        // each quarter's sums, [quarter][column][row] fp32, this warpgroup's
        // half of the columns in two rounds; every warp adds up a quarter of
        // a round's columns
        constexpr int CR = D / 4;
        float* x = reinterpret_cast<float*>(smem + C::OFF_Q) + st * 4 * CR * 32 + lane;
        const float f0 = it.nb > 0 && l != 0.0f ? w0 * inv : 0.0f;
        const float f1 = second && l != 0.0f ? w1 * inv : 0.0f;
        auto meet = [&]() -> bool {  // all 8 warps
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(C::B_X));
          return lane0_wait(bar(C::B_X), meets++ & 1);
        };
#pragma unroll 1
        for (int round = 0; round < 2 && ok; ++round) {
          if (round > 0) ok = meet();
          if (!ok) break;
          const int col = st * (D / 2) + round * CR;
          seq_few_put<D>(tmem + lane_base + C::O_COL, col, x + quad * CR * 32, f0, f1);
          ok = meet();
          if (ok && exists)
            seq_few_take<D, T>(x + quad * (CR / 4) * 32, static_cast<T*>(p.o) + tok_row * D + col + quad * (CR / 4),
                               whole ? nullptr
                                     : p.part_o + (static_cast<size_t>(slot) * 256 + lane) * D + col +
                                           quad * (CR / 4));
        }
        // (the copies that refill Q's place follow these reads and writes)
        ptx::fence_proxy_async_smem();
        if (!ok) break;
      } else if (active) {
#pragma unroll 1
        for (int c = c_lo; c < c_hi; ++c) {
          uint32_t r[32];
          if (cnt > 0 || one) {
            ptx::tmem_ld32(tmem + lane_base + C::O_COL + (one ? 0 : st * D) + 32 * c, r);
            ptx::tmem_wait_ld();
          }
          if (second) {
            uint32_t r2[32];
            ptx::tmem_ld32(tmem + lane_base + C::O_COL + D + 32 * c, r2);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              r[j] = __float_as_uint(w0 * __uint_as_float(r[j]) + w1 * __uint_as_float(r2[j]));
          } else if (one) {
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(w0 * __uint_as_float(r[j]));
          }
#pragma unroll
          for (int j = 0; j < 32; ++j)
            r[j] = l == 0.0f ? 0u : __float_as_uint(__uint_as_float(r[j]) * inv);
          if (exists) {
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.o) + tok_row * D + 32 * c);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  w[k] = seq_pack2<T>(__uint_as_float(r[8 * j + 2 * k]),
                                      __uint_as_float(r[8 * j + 2 * k + 1]));
                dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
              uint4* dst = reinterpret_cast<uint4*>(
                  p.part_o + (static_cast<size_t>(slot) * 256 + prow) * D + 32 * c);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                dst[j] = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
            }
          }
        }
      }
      if (exists && (st == 0 || !one) && (quad == 0 || !few)) {
        if (whole) p.lse[tok_row] = lse2 * 0.6931471805599453f;
        else p.part_lse[static_cast<size_t>(slot) * 256 + prow] = lse2;
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(C::B_OFREE));
    }
    if (!ok) fail();
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == C::WARP_MMA) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Joins the partials of the items that ranges cut: CTA c looks after the item
// that begins in range c and goes on behind it. o = sum_i w_i o_i / sum_i w_i,
// w_i = 2^(lse_i - max), in the order of the ranges.
template <int D, typename T>
__global__ void __launch_bounds__(256) blasst_seq_join_kernel(const SeqAttnParams p) {
  const int c = blockIdx.x;
  ptx::grid_wait();
  const int4 d = p.part_desc[2 * c];
  if (d.x < 0) return;
  const int last = p.part_desc[2 * c + 1].x;
  const int lane = threadIdx.x & 31;
  constexpr int V = D / 32;  // columns per lane
  // rows beyond the item's tokens have no place in o (few rows: rt_few < rt,
  // but the tokens that exist are packed the same)
  const int rows = d.w ? 128 : 256;
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < rows; r += gridDim.y * 8) {
    const int tok = (r >> 7) * p.rt + (r & 127) / p.g;
    if ((r & 127) >= p.g * p.rt || tok >= d.y) continue;
    auto row_of = [&](int k) -> size_t { return static_cast<size_t>(2 * k + (k == c ? 1 : 0)) * 256 + r; };
    float m = -INFINITY, x = -INFINITY;
    for (int k0 = c; k0 <= last; k0 += 32) {  // one part per lane
      x = k0 + lane <= last ? p.part_lse[row_of(k0 + lane)] : -INFINITY;
      float most = x;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, s));
      m = fmaxf(m, most);
    }
    float l = 0.0f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    for (int k0 = c; k0 <= last; k0 += 32) {
      if (last - c >= 32) x = k0 + lane <= last ? p.part_lse[row_of(k0 + lane)] : -INFINITY;
      const float own = x == -INFINITY ? 0.0f : ptx::ex2(x - m);
      const int n = min(32, last - k0 + 1);
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        const float w = __shfl_sync(0xffffffffu, own, k);
        const float* src = p.part_o + row_of(k0 + k) * D + lane * V;
        l += w;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = w == 0.0f ? acc[v] : fmaf(w, src[v], acc[v]);
      }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const long long out = static_cast<long long>(d.x + tok) * p.Hq + d.z * p.g + (r & 127) % p.g;
    uint32_t w2[V / 2];
#pragma unroll
    for (int v = 0; v < V / 2; ++v) w2[v] = seq_pack2<T>(acc[2 * v] * inv, acc[2 * v + 1] * inv);
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(p.o) + out * D) + lane * (V / 2);
#pragma unroll
    for (int v = 0; v < V / 2; ++v) dst[v] = w2[v];
    if (lane == 0) p.lse[out] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
}

}  // namespace blasst
