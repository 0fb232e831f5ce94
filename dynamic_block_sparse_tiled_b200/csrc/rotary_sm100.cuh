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
// keeps its place within the head, so its sines stay in registers while it
// walks the heads, 16 bytes per load where sizes and strides allow.
// Bound by memory: each value is read once and written once.
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
  int hb;
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

template <typename T>
__device__ __forceinline__ float rot_load(T v) {
  return static_cast<float>(v);
}

template <typename T, int N>
struct alignas(sizeof(T) * N) RotVec {
  T e[N];
};

// One place within the heads of one token: turn (or copy) and store.
// v < npair: vector v of the pairs; else a vector of the dims behind rot.
template <typename T, int VEC>
struct RotaryLane {
  float2 cs[VEC];
  int v;
  bool turn;

  __device__ __forceinline__ void set(const float2* row, int v_, int rot, bool interleaved) {
    v = v_;
    if (interleaved) {
      // VEC values are VEC / 2 pairs; a scalar step takes one pair
      constexpr int NP = VEC == 1 ? 1 : VEC / 2;
      turn = v * NP < rot / 2;
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (turn) cs[i] = row[v * NP + i];
    } else {
      turn = v * VEC < rot / 2;
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (turn) cs[i] = row[v * VEC + i];
    }
  }

  __device__ __forceinline__ void apply(const T* x, T* y, int rot, bool interleaved) const {
    if (interleaved) {
      constexpr int N = VEC == 1 ? 2 : VEC;
      if (turn) {
        T in[N], out[N];
        if constexpr (VEC == 1) {
          in[0] = x[2 * v];
          in[1] = x[2 * v + 1];
        } else {
          *reinterpret_cast<RotVec<T, VEC>*>(in) = reinterpret_cast<const RotVec<T, VEC>*>(x)[v];
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float a = rot_load(in[2 * i]), b = rot_load(in[2 * i + 1]);
          out[2 * i] = static_cast<T>(a * cs[i].x - b * cs[i].y);
          out[2 * i + 1] = static_cast<T>(a * cs[i].y + b * cs[i].x);
        }
        if constexpr (VEC == 1) {
          y[2 * v] = out[0];
          y[2 * v + 1] = out[1];
        } else {
          reinterpret_cast<RotVec<T, VEC>*>(y)[v] = *reinterpret_cast<RotVec<T, VEC>*>(out);
        }
      } else if constexpr (VEC == 1) {
        const int i = rot + (v - rot / 2);  // one value behind rot
        y[i] = x[i];
      } else {
        reinterpret_cast<RotVec<T, VEC>*>(y)[v] = reinterpret_cast<const RotVec<T, VEC>*>(x)[v];
      }
    } else {
      using V = RotVec<T, VEC>;
      if (turn) {
        const V a = *reinterpret_cast<const V*>(x + v * VEC);
        const V b = *reinterpret_cast<const V*>(x + rot / 2 + v * VEC);
        V c, e;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float p = rot_load(a.e[i]), q = rot_load(b.e[i]);
          c.e[i] = static_cast<T>(p * cs[i].x - q * cs[i].y);
          e.e[i] = static_cast<T>(p * cs[i].y + q * cs[i].x);
        }
        *reinterpret_cast<V*>(y + v * VEC) = c;
        *reinterpret_cast<V*>(y + rot / 2 + v * VEC) = e;
      } else {
        const int i = rot + (v - rot / 2 / VEC) * VEC;
        *reinterpret_cast<V*>(y + i) = *reinterpret_cast<const V*>(x + i);
      }
    }
  }
};

// Places within a head: pairs (of vectors), then the vectors behind rot.
__host__ __device__ __forceinline__ int rotary_places(int d, int rot, bool interleaved, int vec) {
  if (interleaved) return vec == 1 ? rot / 2 + (d - rot) : d / vec;
  return rot / 2 / vec + (d - rot) / vec;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(256) blasst_rotary_kernel(const RotaryParams p) {
  extern __shared__ float2 cs_rows[];  // [tb][rot / 2]
  const int half = p.rot / 2;
  const long long tokens = static_cast<long long>(p.B) * p.L;
  const long long t0 = static_cast<long long>(blockIdx.x) * p.tb;
  const int nt = static_cast<int>(min(static_cast<long long>(p.tb), tokens - t0));
  for (int i = threadIdx.x; i < nt * half; i += 256) {
    const long long t = t0 + i / half;
    const int b = static_cast<int>(t / p.L), l = static_cast<int>(t % p.L);
    double pos = l;
    if (p.pos) {
      const long long at = b * p.pos_sb + l;
      pos = p.pos64 ? static_cast<double>(static_cast<const long long*>(p.pos)[at])
                    : static_cast<double>(static_cast<const int*>(p.pos)[at]);
    }
    cs_rows[i] = rotary_cs(pos, p.freq[i % half], p.sign, p.mscale);
  }
  __syncthreads();
  const bool il = p.interleaved != 0;
  const int nv = rotary_places(p.d, p.rot, il, VEC);
  const int nvb = min(nv, 256);
  const int groups = 256 / nvb;
  const int group = threadIdx.x / nvb;
  if (group >= groups) return;
  const int h_end = min(p.H, static_cast<int>(blockIdx.y + 1) * p.hb);
  for (int i = 0; i < nt; ++i) {
    const long long t = t0 + i;
    const long long b = t / p.L, l = t % p.L;
    const T* x = static_cast<const T*>(p.x) + b * p.x_sb + l * p.x_st;
    T* y = static_cast<T*>(p.y) + b * p.y_sb + l * p.y_st;
    for (int v = threadIdx.x % nvb; v < nv; v += nvb) {
      RotaryLane<T, VEC> lane;
      lane.set(cs_rows + i * half, v, p.rot, il);
#pragma unroll 4
      for (int h = blockIdx.y * p.hb + group; h < h_end; h += groups)
        lane.apply(x + h * p.x_sh, y + h * p.y_sh, p.rot, il);
    }
  }
}

// One token per block row: q's heads, then k's, then v's.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) blasst_append_kernel(const AppendParams p) {
  extern __shared__ float2 cs_rows[];  // [rot / 2]
  const int t = blockIdx.x;
  const int half = p.rot / 2;
  // the token's sequence: sequences that end at or before it
  int s = 0;
  for (int i0 = 0; i0 < p.n_seq; i0 += 256) {
    const int i = i0 + threadIdx.x;
    const int c = __syncthreads_count(i < p.n_seq && p.cu_q[i + 1] <= t);
    s += c;
    if (c < 256) break;
  }
  if (s >= p.n_seq || p.cu_q[s] > t) return;  // behind the last sequence, or before the first
  const int q0 = p.cu_q[s], q1 = p.cu_q[s + 1], kv = p.kv_lens[s];
  const long long pos = static_cast<long long>(kv) - (q1 - t);
  const long long cap = static_cast<long long>(p.table_width) * p.page_size;
  bool place = q0 >= 0 && pos >= 0 && pos < cap;
  int page = 0;
  if (place) {
    page = p.table[static_cast<long long>(s) * p.table_stride + pos / p.page_size];
    place = page >= 0 && page < p.n_pages;
  }
  if (!place && threadIdx.x == 0) seq_record_error(p.err, BLASST_EINDEX);
  for (int i = threadIdx.x; i < half; i += 256)
    cs_rows[i] = rotary_cs(static_cast<double>(pos), p.freq[i], 1.0f, p.mscale);
  __syncthreads();
  const bool il = p.interleaved != 0;
  const int nv = rotary_places(p.d, p.rot, il, VEC);
  const int nvb = min(nv, 256);
  const int groups = 256 / nvb;
  const int group = threadIdx.x / nvb;
  if (group >= groups) return;
  const int hq = p.q ? p.Hq : 0;
  const int heads = hq + 2 * p.Hkv;
  const int h_end = min(heads, static_cast<int>(blockIdx.y + 1) * p.hb);
  const long long row = pos % p.page_size;
  for (int v = threadIdx.x % nvb; v < nv; v += nvb) {
    RotaryLane<T, VEC> lane;
    lane.set(cs_rows, v, p.rot, il);
    for (int hh = blockIdx.y * p.hb + group; hh < h_end; hh += groups) {
      if (hh < hq) {
        lane.apply(static_cast<const T*>(p.q) + t * p.q_st + hh * p.q_sh,
                   static_cast<T*>(p.q_out) + t * p.qo_st + hh * p.qo_sh, p.rot, il);
      } else if (place) {
        const int h = (hh - hq) % p.Hkv;
        if (hh - hq < p.Hkv) {
          lane.apply(static_cast<const T*>(p.k) + t * p.k_st + h * p.k_sh,
                     static_cast<T*>(p.k_pages) + page * p.kp_sp + row * p.kp_st + h * p.kp_sh,
                     p.rot, il);
        } else {
          // v is copied: the same places, nothing turned
          const T* x = static_cast<const T*>(p.v) + t * p.v_st + h * p.v_sh;
          T* y = static_cast<T*>(p.v_pages) + page * p.vp_sp + row * p.vp_st + h * p.vp_sh;
          RotaryLane<T, VEC> copy;
          copy.v = v;
          copy.turn = false;
          if (lane.turn) {
            // the place's own values: a pair (interleaved) or two vectors
            if (il && VEC == 1) {
              y[2 * v] = x[2 * v];
              y[2 * v + 1] = x[2 * v + 1];
            } else {
              using V = RotVec<T, VEC>;
              *reinterpret_cast<V*>(y + v * VEC) = *reinterpret_cast<const V*>(x + v * VEC);
              if (!il)
                *reinterpret_cast<V*>(y + half + v * VEC) =
                    *reinterpret_cast<const V*>(x + half + v * VEC);
            }
          } else {
            copy.apply(x, y, p.rot, il);
          }
        }
      }
    }
  }
}

}  // namespace blasst
