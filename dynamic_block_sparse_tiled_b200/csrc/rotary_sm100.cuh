// rotary_sm100.cuh - rotary position embedding, and the write of new tokens
// into a paged KV cache with q and k turned on the way.
//
// Pair i of a head (i < rot / 2) turns by the angle a = position * f_i:
//   y_a = (x_a cos a - x_b sin a) s,   y_b = (x_a sin a + x_b cos a) s,
// (a, b) = (i, i + rot / 2) ("half") or (2 i, 2 i + 1) (interleaved); dims from
// rot on are copied. The backward pass is the transposed turn (sin negated).
//
// The angle is formed in 64 bits and reduced to [-pi, pi] there, in half
// turns (a far position times a fast frequency loses all of its fraction in
// 32 bits); sine and cosine of the reduced angle in 32 bits. One block takes a
// few tokens: it forms each (token, pair) once, and every head uses it. A thread
// keeps its token and its place within the head, so its sines stay in registers
// while it walks the heads, four at a time, 16 bytes per load where sizes and
// strides allow; its first loads are on their way while the angles are formed.
// Bound by memory: each value is read once and written once. 32768 tokens of 32
// heads of 128, bf16: 96 us, 5.6 TB/s (86 % of a copy's rate), at three blocks
// per SM; 106 us at the two that the compiler's own choice of registers left.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/blasst.h"
#include "attn_seq_sm100.cuh"

namespace blasst {

struct RotaryParams {
  const void* x;
  void* y;
  const void* pos;       // null: the token's index in its row
  const double* freq;    // [rot / 2], radians per position
  long long x_sb, x_st, x_sh, y_sb, y_st, y_sh, pos_sb;
  int pos64;
  int B, L, H, d, rot;
  int interleaved;
  float sign, mscale;
  int tb;  // tokens per block
  int hb;  // heads per block
};

struct AppendParams {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_pages;
  void* v_pages;
  long long q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh;
  long long kp_sp, kp_st, kp_sh, vp_sp, vp_st, vp_sh;
  const int* table;
  long long table_stride;
  int table_width, page_size, n_pages;
  const int* kv_lens;
  const int* cu_q;
  int n_seq, T, Hq, Hkv, d, rot, interleaved;
  const double* freq;
  float mscale;
  int tb;  // tokens per block
  int hb;  // heads per block
  int* err;
};

// (cos, sin) of position * f, scaled; `f` in radians.
__device__ __forceinline__ float2 rotary_cs(double position, double f, float sign, float mscale) {
  double h = position * f * 0.31830988618379067154;  // 1 / pi: half turns
  h -= 2.0 * rint(0.5 * h);
  float sn, cs;
  sincospif(static_cast<float>(h), &sn, &cs);
  return make_float2(cs * mscale, sn * mscale * sign);
}

// N values as they lie in memory, kept as words until they are used (16-bit
// values one to a register took 120 registers, and 141 us where words take 106).
template <typename T, int N>
struct alignas(sizeof(T) * N) RotVec {
  static constexpr int kWords = static_cast<int>(sizeof(T)) * N / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else if constexpr (SeqType<T>::kFormat == 1)
      return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i / 2]));
      return i & 1 ? f.y : f.x;
    }
  }
  // values i, i + 1 (i even)
  __device__ __forceinline__ void put2(int i, float x, float y) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(x);
      w[i + 1] = __float_as_uint(y);
    } else {
      w[i / 2] = seq_pack2<T>(x, y);
    }
  }
};
template <typename T>
struct alignas(sizeof(T)) RotVec<T, 1> {
  T e;
  __device__ __forceinline__ float get(int) const { return static_cast<float>(e); }
};

// One place within a head: a pair of vectors (half), a vector of pairs
// (interleaved), or a vector of the dims behind rot.
// v < npair: vector v of the pairs; else a vector of the dims behind rot.
template <typename T, int VEC, bool IL>
struct RotaryPlace {
  using V = RotVec<T, VEC>;
  static constexpr int NP = IL && VEC > 1 ? VEC / 2 : VEC;  // pairs
  static constexpr bool kTwo = !IL || VEC == 1;             // a pair's values come by two loads
  int at, at2, pair;  // offsets in the head, first pair; pair < 0: not turned

  __device__ __forceinline__ RotaryPlace(int v, int rot) {
    const int half = rot / 2;
    const bool turn = v * NP < half;
    pair = turn ? v * NP : -1;
    if (turn) {
      at = IL ? (VEC == 1 ? 2 * v : v * VEC) : v * VEC;
      at2 = IL ? at + 1 : half + v * VEC;
    } else {
      at = rot + (v - half / NP) * VEC;
      at2 = at;
    }
  }
  __device__ __forceinline__ void load(const T* x, V& a, V& b) const {
    a = *reinterpret_cast<const V*>(x + at);
    if constexpr (kTwo) b = *reinterpret_cast<const V*>(x + at2);
  }
  __device__ __forceinline__ void store(T* y, const V& a, const V& b) const {
    *reinterpret_cast<V*>(y + at) = a;
    if constexpr (kTwo)
      if (pair >= 0) *reinterpret_cast<V*>(y + at2) = b;
  }
  // cs: (cos, sin) of the place's pairs
  __device__ __forceinline__ void turn(const float2 (&cs)[NP], V& a, V& b) const {
    if constexpr (VEC == 1) {
      const float u = a.get(0), w = b.get(0);
      a.e = static_cast<T>(u * cs[0].x - w * cs[0].y);
      b.e = static_cast<T>(u * cs[0].y + w * cs[0].x);
    } else if constexpr (IL) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float u = a.get(2 * i), w = a.get(2 * i + 1);
        a.put2(2 * i, u * cs[i].x - w * cs[i].y, u * cs[i].y + w * cs[i].x);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; i += 2) {
        const float u0 = a.get(i), w0 = b.get(i), u1 = a.get(i + 1), w1 = b.get(i + 1);
        a.put2(i, u0 * cs[i].x - w0 * cs[i].y, u1 * cs[i + 1].x - w1 * cs[i + 1].y);
        b.put2(i, u0 * cs[i].y + w0 * cs[i].x, u1 * cs[i + 1].y + w1 * cs[i + 1].x);
      }
    }
  }
};

// Places within a head: pairs (of vectors), then the vectors behind rot.
__host__ __device__ __forceinline__ int rotary_places(int d, int rot, bool interleaved, int vec) {
  if (interleaved) return vec == 1 ? rot / 2 + (d - rot) : d / vec;
  return rot / 2 / vec + (d - rot) / vec;
}

constexpr int kRotaryAhead = 4;  // heads a thread has on their way

template <typename T, int VEC, bool IL>
__global__ void __launch_bounds__(256, 3) blasst_rotary_kernel(const RotaryParams p) {
  using P = RotaryPlace<T, VEC, IL>;
  extern __shared__ float2 cs_rows[];  // [tb][rot / 2]
  const int half = p.rot / 2;
  const long long tokens = static_cast<long long>(p.B) * p.L;
  const long long t0 = static_cast<long long>(blockIdx.x) * p.tb;
  const int nt = static_cast<int>(min(static_cast<long long>(p.tb), tokens - t0));
  const int nv = rotary_places(p.d, p.rot, IL, VEC);
  const int nvb = min(nv, 256);
  const int lanes = 256 / nvb / p.tb;  // heads of a token at the same time
  const int group = threadIdx.x / nvb;
  const int row = group / lanes, sub = group % lanes;
  const bool takes = row < nt;
  const long long t = t0 + min(row, nt - 1);
  const long long bt = p.B == 1 ? 0 : t / p.L, l = t - bt * p.L;
  const T* x = static_cast<const T*>(p.x) + bt * p.x_sb + l * p.x_st;
  T* y = static_cast<T*>(p.y) + bt * p.y_sb + l * p.y_st;
  const int h_end = min(p.H, static_cast<int>(blockIdx.y + 1) * p.hb);
  bool formed = false;
  for (int v = threadIdx.x % nvb; v < nv || !formed; v += nvb) {
    const P place(min(v, nv - 1), p.rot);
    const bool mine = takes && v < nv;
    float2 cs[P::NP];
    bool first = true;
    for (int h0 = blockIdx.y * p.hb + sub; h0 < h_end || !formed; h0 += kRotaryAhead * lanes) {
      typename P::V a[kRotaryAhead], b[kRotaryAhead];
#pragma unroll
      for (int k = 0; k < kRotaryAhead; ++k) {
        const int h = h0 + k * lanes;
        if (mine && h < h_end) place.load(x + h * p.x_sh, a[k], b[k]);
      }
      if (!formed) {
        for (int i = threadIdx.x; i < nt * half; i += 256) {
          const long long ti = t0 + i / half;
          const long long bi = p.B == 1 ? 0 : ti / p.L, li = ti - bi * p.L;
          double pos = static_cast<double>(li);
          if (p.pos) {
            const long long at = bi * p.pos_sb + li;
            pos = p.pos64 ? static_cast<double>(static_cast<const long long*>(p.pos)[at])
                          : static_cast<double>(static_cast<const int*>(p.pos)[at]);
          }
          cs_rows[i] = rotary_cs(pos, p.freq[i % half], p.sign, p.mscale);
        }
        __syncthreads();
        formed = true;
      }
      if (first && place.pair >= 0) {
#pragma unroll
        for (int i = 0; i < P::NP; ++i) cs[i] = cs_rows[min(row, nt - 1) * half + place.pair + i];
      }
      first = false;
#pragma unroll
      for (int k = 0; k < kRotaryAhead; ++k) {
        const int h = h0 + k * lanes;
        if (!mine || h >= h_end) continue;
        if (place.pair >= 0) place.turn(cs, a[k], b[k]);
        place.store(y + h * p.y_sh, a[k], b[k]);
      }
    }
  }
}

// A few tokens per block: of each q's heads, then k's, then v's. A token's way to
// its page (sequence, length, table entry, angles) is a chain of dependent reads
// of about 3 us, so a block takes as many tokens as there are to keep it busy:
// 2560 tokens of 48 heads of 128, fp16, on warm inputs: 12.5 us (5.0 TB/s, 78 % of
// a copy's rate) with four, 14.3 us with one; on changing ones 18.4 us with eight
// (3.4 TB/s) and 18.5 us with four, which is no difference.
constexpr int kAppendTokens = 8;  // most tokens of a block, one warp each to find its place

template <typename T, int VEC, bool IL>
__global__ void __launch_bounds__(256) blasst_append_kernel(const AppendParams p) {
  using P = RotaryPlace<T, VEC, IL>;
  extern __shared__ float2 cs_rows[];  // [tb][rot / 2]
  struct Where {
    long long page, row;
    int owned, placed, pos;
  };
  __shared__ Where where[kAppendTokens];
  const int t0 = blockIdx.x * p.tb;
  const int nt = min(p.tb, p.T - t0);
  const int half = p.rot / 2;
  const int nv = rotary_places(p.d, p.rot, IL, VEC);
  const int nvb = min(nv, 256);
  const int lanes = 256 / nvb / p.tb;  // heads of a token at the same time
  const int group = threadIdx.x / nvb;
  const int tok = min(group / lanes, nt - 1), sub = group % lanes;
  const bool takes = group / lanes < nt;
  const long long t = t0 + tok;
  const int hq = p.q ? p.Hq : 0;
  const int h_end = min(hq + 2 * p.Hkv, static_cast<int>(blockIdx.y + 1) * p.hb);
  const T* q = static_cast<const T*>(p.q) + t * p.q_st;
  const T* k = static_cast<const T*>(p.k) + t * p.k_st;
  const T* v = static_cast<const T*>(p.v) + t * p.v_st;
  T* q_out = static_cast<T*>(p.q_out) + t * p.qo_st;
  bool formed = false;
  Where at{};
  for (int place_i = threadIdx.x % nvb; place_i < nv || !formed; place_i += nvb) {
    const P place(min(place_i, nv - 1), p.rot);
    bool mine = takes && place_i < nv;
    float2 cs[P::NP];
    bool first = true;
    for (int h0 = blockIdx.y * p.hb + sub; h0 < h_end || !formed; h0 += kRotaryAhead * lanes) {
      typename P::V a[kRotaryAhead], b[kRotaryAhead];
#pragma unroll
      for (int u = 0; u < kRotaryAhead; ++u) {
        const int h = h0 + u * lanes;
        if (!mine || h >= h_end) continue;
        place.load(h < hq ? q + h * p.q_sh : h < hq + p.Hkv ? k + (h - hq) * p.k_sh : v + (h - hq - p.Hkv) * p.v_sh,
                   a[u], b[u]);
      }
      if (!formed) {
        const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (w < nt) {
          // the token's sequence: sequences that end at or before it
          const int tw = t0 + w;
          int s = 0;
          for (int j0 = 0; j0 < p.n_seq; j0 += 32) {
            const int j = j0 + lane;
            const int c = __popc(__ballot_sync(0xffffffffu, j < p.n_seq && p.cu_q[j + 1] <= tw));
            s += c;
            if (c < 32) break;
          }
          if (lane == 0) {
            Where x{};
            x.owned = s < p.n_seq && p.cu_q[s] <= tw;  // else behind the last sequence, or before the first
            if (x.owned) {
              const int q0 = p.cu_q[s], q1 = p.cu_q[s + 1], kv = p.kv_lens[s];
              const long long pos = static_cast<long long>(kv) - (static_cast<long long>(q1) - tw);
              const long long cap = static_cast<long long>(p.table_width) * p.page_size;
              x.placed = q0 >= 0 && q1 <= p.T && pos >= 0 && pos < cap;
              // (a position is below 2^31: it counts from a 32-bit length)
              x.pos = static_cast<int>(pos);
              if (x.placed) {
                const uint32_t in_table = static_cast<uint32_t>(x.pos) / static_cast<uint32_t>(p.page_size);
                x.page = p.table[static_cast<long long>(s) * p.table_stride + in_table];
                x.row = x.pos - static_cast<long long>(in_table) * p.page_size;
                x.placed = x.page >= 0 && x.page < p.n_pages;
              }
              if (!x.placed) seq_record_error(p.err, BLASST_EINDEX);
            }
            where[w] = x;
          }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < nt * half; i += 256)
          cs_rows[i] = rotary_cs(static_cast<double>(where[i / half].pos), p.freq[i % half], 1.0f, p.mscale);
        __syncthreads();
        formed = true;
        at = where[tok];
      }
      mine = mine && at.owned;
      if (first && place.pair >= 0) {
#pragma unroll
        for (int i = 0; i < P::NP; ++i) cs[i] = cs_rows[tok * half + place.pair + i];
      }
      first = false;
#pragma unroll
      for (int u = 0; u < kRotaryAhead; ++u) {
        const int h = h0 + u * lanes;
        if (!mine || h >= h_end) continue;
        const bool is_v = h >= hq + p.Hkv;
        if (place.pair >= 0 && !is_v) place.turn(cs, a[u], b[u]);
        if (h < hq) {
          place.store(q_out + h * p.qo_sh, a[u], b[u]);
        } else if (at.placed) {
          place.store(is_v ? static_cast<T*>(p.v_pages) + at.page * p.vp_sp + at.row * p.vp_st + (h - hq - p.Hkv) * p.vp_sh
                           : static_cast<T*>(p.k_pages) + at.page * p.kp_sp + at.row * p.kp_st + (h - hq) * p.kp_sh,
                      a[u], b[u]);
        }
      }
    }
  }
}

}  // namespace blasst
