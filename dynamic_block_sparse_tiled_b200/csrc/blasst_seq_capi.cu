// blasst_seq_capi.cu - C ABI of the operators over sequences of different
// lengths (include/blasst.h): argument checks, tensor maps, launch rules.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/blasst.h"
#include "attn_seq_bwd_sm100.cuh"
#include "attn_seq_sm100.cuh"
#include "capi_internal.h"
#include "rotary_sm100.cuh"

namespace {

using blasst::capi::cuda_status;
using blasst::capi::encode_tiled;
using blasst::capi::error_word;
using blasst::capi::kTimeoutNs;

constexpr int kMaxDevices = 64;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// SMs of the current device (a host-side query, kept per device; host threads may
// find it at the same time).
int sm_count() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  int n = dev < kMaxDevices ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < kMaxDevices) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// 4-D map (d, rows, heads or groups, outer), 128-byte swizzle, zero fill
// outside. Strides in elements of 2 bytes.
bool make_map4(CUtensorMap* map, const void* base, int dtype, const long long (&dim)[4],
               const long long (&stride)[3], int box1, int box2) {
  cuuint64_t dims[4], strides[3];
  for (int i = 0; i < 4; ++i) dims[i] = static_cast<cuuint64_t>(dim[i] > 0 ? dim[i] : 1);
  // the stride of a dimension of one entry is never used, but has to be valid
  for (int i = 0; i < 3; ++i)
    strides[i] = dims[i + 1] == 1 ? 16 : static_cast<cuuint64_t>(stride[i]) * 2;
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2), 1};
  const auto dt = dtype == BLASST_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return encode_tiled(map, dt, 4, const_cast<void*>(base), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// A stride a tensor map can hold: positive, a multiple of 16 bytes, < 2^40.
bool map_stride(long long elems) { return elems > 0 && elems % 8 == 0 && elems < (1ll << 39); }

size_t seq_workspace(int sms, int d) {
  return static_cast<size_t>(sms) * (2 * 256 * (static_cast<size_t>(d) + 1) * 4 + 32);
}

// The register split of a kernel waits for registers the launch must have:
// refused (not run) if a build gave the kernel fewer.
template <typename K>
int check_regs(K kernel, int regs, std::atomic<int>& known) {
  int have = known.load(std::memory_order_relaxed);
  if (have == 0) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return cuda_status(e);
    have = fa.numRegs;
    known.store(have, std::memory_order_relaxed);
  }
  return have >= regs ? BLASST_OK : BLASST_EUNSUPPORTED;
}

// A launch that may begin while the kernel before it runs; the kernel waits for
// that one's end itself.
template <typename K, typename... A>
cudaError_t launch_early(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = &early;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, args...);
}

template <int D, typename T, bool FEW>
int launch_seq(const CUtensorMap& mq, const CUtensorMap& mq_few, const CUtensorMap& mk,
               const CUtensorMap& mv, const blasst::SeqAttnParams& p, int sms, cudaStream_t stream) {
  using C = blasst::SeqAttnCfg<D, FEW>;
  auto kernel = blasst::blasst_seq_attn_kernel<D, T, FEW>;
  static std::atomic<int> regs{0};  // of this instantiation
  if (const int rc = check_regs(kernel, C::REGS, regs)) return rc;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return cuda_status(e);
  const bool shared_list = p.n_tiles == 0;
  const unsigned grid =
      shared_list || p.next ? static_cast<unsigned>(sms) : static_cast<unsigned>(p.n_tiles) * p.Hkv;
  if (p.next) {
    e = cudaMemsetAsync(p.next, 0, sizeof(int), stream);
    if (e != cudaSuccess) return cuda_status(e);
  }
  kernel<<<grid, C::NTHREADS, C::SMEM_BYTES, stream>>>(mq, mq_few, mk, mv, p);
  int rc = cuda_status(cudaGetLastError());
  if (rc != BLASST_OK || !shared_list) return rc;
  return cuda_status(launch_early(blasst::blasst_seq_join_kernel<D, T>, dim3(grid, 4), 256, 0, stream, p));
}

template <int D, typename T>
int launch_seq_few(bool few, const CUtensorMap& mq, const CUtensorMap& mq_few, const CUtensorMap& mk,
                   const CUtensorMap& mv, const blasst::SeqAttnParams& p, int sms, cudaStream_t stream) {
  return few ? launch_seq<D, T, true>(mq, mq_few, mk, mv, p, sms, stream)
             : launch_seq<D, T, false>(mq, mq_few, mk, mv, p, sms, stream);
}

constexpr long long kSeqFewKeys = 1024;

// What the packed and the paged call share; `p` holds the keys' side already.
int run_seq(blasst::SeqAttnParams& p, const void* q, long long q_st, long long q_sh, int d,
            float scale, int dtype, const CUtensorMap& mk, const CUtensorMap& mv,
            long long most_keys, void* workspace, int sms, void* stream) {
  p.rt = 128 / p.g;
  // The kernel for few rows when the sequences have up to 32 rows on average.
  // Whole items once the tiles fill the GPU several times (their order then shares
  // K and V in L2), or if no sequence can have many keys (nothing worth cutting,
  // and no second kernel). Fewer tiles, or mostly single tokens: the shared list,
  // which cuts long rows of key blocks between SMs. A whole item is never cut, so a
  // few tokens over a very long cache beside many prompt tokens take as long as one
  // CTA needs for them (8192 tokens of 64 / 8 heads of 128 and one over 262144 keys:
  // 3.0 ms in one call, 1.04 and 0.18 in two).
  p.rt_few = p.g <= 32 ? 32 / p.g : 0;
  const bool few = p.rt_few > 0 && static_cast<long long>(p.Tq) * p.g <= 32ll * p.n_seq;
  p.it_tok = few ? p.rt : 2 * p.rt;
  const long long full = static_cast<long long>(p.Tq) / p.it_tok;
  const long long tiles = full + p.n_seq;  // places (seq_place)
  const bool single = full * p.Hkv >= 8ll * sms || most_keys <= kSeqFewKeys;
  p.n_tiles = single && tiles * p.Hkv < 0x7fffffffll ? static_cast<int>(tiles) : 0;
  // Several whole items per SM: a resident grid takes them from a list, so that an
  // item's end and the next one's loads overlap (a CTA of its own cost each item
  // about 4 us of set-up; the list costs its clearing, 2 us); else a CTA each.
  p.next = p.n_tiles != 0 && static_cast<long long>(p.n_tiles) * p.Hkv > 2ll * sms ? static_cast<int*>(workspace) : nullptr;
  const size_t rows = static_cast<size_t>(sms) * 2 * 256;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = p.part_o + rows * d;
  p.part_desc = reinterpret_cast<int4*>(p.part_lse + rows);
  const double sc = scale > 0.0f ? static_cast<double>(scale) : 1.0 / std::sqrt(static_cast<double>(d));
  p.scale_log2 = static_cast<float>(sc * 1.4426950408889634);
  p.timeout_ns = kTimeoutNs;
  CUtensorMap mq, mq_few;
  if (!make_map4(&mq, q, dtype, {d, p.g, p.Tq, p.Hkv}, {q_sh, q_st, q_sh * p.g}, p.g, p.rt) ||
      !make_map4(&mq_few, q, dtype, {d, p.g, p.Tq, p.Hkv}, {q_sh, q_st, q_sh * p.g}, p.g,
                 std::max(1, p.rt_few)))
    return BLASST_ECUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == BLASST_BF16)
    return d == 128 ? launch_seq_few<128, __nv_bfloat16>(few, mq, mq_few, mk, mv, p, sms, s)
                    : launch_seq_few<64, __nv_bfloat16>(few, mq, mq_few, mk, mv, p, sms, s);
  return d == 128 ? launch_seq_few<128, __half>(few, mq, mq_few, mk, mv, p, sms, s)
                  : launch_seq_few<64, __half>(few, mq, mq_few, mk, mv, p, sms, s);
}

int check_heads(int n_seq, int Tq, int Hq, int Hkv, int d, int dtype) {
  if (n_seq < 0 || Tq < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return BLASST_EINVAL;
  if (Hkv > 65535 || n_seq > (1 << 24)) return BLASST_EINVAL;
  if (d != 64 && d != 128) return BLASST_EUNSUPPORTED;
  if (Hq / Hkv > 128) return BLASST_EUNSUPPORTED;
  if (dtype != BLASST_BF16 && dtype != BLASST_FP16) return BLASST_EUNSUPPORTED;
  return BLASST_OK;
}

// Two words per query row, and 16 bytes per KV head that keep a call without
// query rows from asking for none.
size_t bwd_workspace(int Tq, int Hq, int Hkv) {
  return static_cast<size_t>(Hkv) * 16 + static_cast<size_t>(Tq) * Hq * sizeof(float2);
}

template <int D, typename T>
int launch_seq_bwd(const CUtensorMap& mq, const CUtensorMap& mdo, const CUtensorMap& mk,
                   const CUtensorMap& mv, const blasst::SeqBwdParams& p,
                   const blasst::SeqBwdRowsParams& r, cudaStream_t stream) {
  using C = blasst::SeqBwdCfg<D>;
  auto kernel = blasst::blasst_seq_bwd_kernel<D, T>;
  static std::atomic<int> regs{0};  // of this instantiation
  if (const int rc = check_regs(kernel, C::REGS, regs)) return rc;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return cuda_status(e);
  if (r.Tq > 0) {
    // places for parts of v (seq_place)
    const int v_blocks = blasst::SeqBwdType<T>::kScaled && r.Tk > 0 ? r.Tk / blasst::kBwdRowsPerBlock + r.n_seq : 0;
    blasst::blasst_seq_bwd_rows_kernel<D, T>
        <<<dim3(static_cast<unsigned>(r.row_blocks + v_blocks), r.Hkv), 256, 0, stream>>>(r);
    const int rc = cuda_status(cudaGetLastError());
    if (rc != BLASST_OK) return rc;
  }
  const unsigned grid = static_cast<unsigned>(p.n_key + p.n_row) * p.Hkv;
  if (r.Tq > 0)
    return cuda_status(launch_early(kernel, dim3(grid), C::NTHREADS, C::SMEM_BYTES, stream, mq, mdo, mk, mv, p));
  kernel<<<grid, C::NTHREADS, C::SMEM_BYTES, stream>>>(mq, mdo, mk, mv, p);
  return cuda_status(cudaGetLastError());
}

int elem_bytes(int dtype) { return dtype == BLASST_FP32 ? 4 : 2; }

// Widest vector (elements) that both sides' base and strides allow.
bool vector_ok(const void* p, const long long* strides, int n, int vec, int bytes) {
  if (!aligned(p, static_cast<uintptr_t>(vec) * bytes)) return false;
  for (int i = 0; i < n; ++i)
    if (strides[i] % vec != 0) return false;
  return true;
}

bool rotary_vec(int d, int rot, bool interleaved, int vec) {
  if (interleaved) return d % vec == 0 && rot % vec == 0;
  return (rot / 2) % vec == 0 && (d - rot) % vec == 0;
}

template <typename T, int VEC>
int launch_rotary(const blasst::RotaryParams& p, dim3 grid, size_t smem, cudaStream_t s) {
  if (p.interleaved) blasst::blasst_rotary_kernel<T, VEC, true><<<grid, 256, smem, s>>>(p);
  else blasst::blasst_rotary_kernel<T, VEC, false><<<grid, 256, smem, s>>>(p);
  return cuda_status(cudaGetLastError());
}

template <typename T, int VEC>
int launch_append(const blasst::AppendParams& p, dim3 grid, size_t smem, cudaStream_t s) {
  if (p.interleaved) blasst::blasst_append_kernel<T, VEC, true><<<grid, 256, smem, s>>>(p);
  else blasst::blasst_append_kernel<T, VEC, false><<<grid, 256, smem, s>>>(p);
  return cuda_status(cudaGetLastError());
}

// Heads per block: all of them, unless few tokens would leave SMs idle.
int heads_per_block(long long blocks, int heads, int places, int sms) {
  const int groups = std::max(1, 256 / std::min(places, 256));
  int split = 1;
  while (blocks * split < 2ll * sms && heads > groups * split) split *= 2;
  return (heads + split - 1) / split;
}

}  // namespace

extern "C" {

int blasst_rotary(const blasst_rotary_args* a) {
  if (!a || !a->x || !a->y || !a->freq) return BLASST_EINVAL;
  if (a->dtype != BLASST_BF16 && a->dtype != BLASST_FP16 && a->dtype != BLASST_FP32)
    return BLASST_EUNSUPPORTED;
  const int eb = elem_bytes(a->dtype);
  if (a->B < 0 || a->L < 0 || a->H < 0 || a->d <= 0 || a->rot < 2 || a->rot > a->d ||
      a->rot % 2 != 0)
    return BLASST_EINVAL;
  if (!(a->scale > 0.0f) || !std::isfinite(a->scale)) return BLASST_EINVAL;
  if (a->d > 1024) return BLASST_EUNSUPPORTED;
  if (!aligned(a->x, eb) || !aligned(a->y, eb) || !aligned(a->freq, 8) ||
      (a->positions && !aligned(a->positions, a->pos64 ? 8 : 4)))
    return BLASST_EINVAL;
  // the same elements by other strides would be read after they are written
  if (a->x == a->y && (a->x_sb != a->y_sb || a->x_sl != a->y_sl || a->x_sh != a->y_sh))
    return BLASST_EINVAL;
  const long long tokens = static_cast<long long>(a->B) * a->L;
  if (tokens == 0 || a->H == 0) return BLASST_OK;
  const int sms = sm_count();
  if (sms == 0) return BLASST_ECUDA;
  blasst::RotaryParams p{};
  p.x = a->x;
  p.y = a->y;
  p.pos = a->positions;
  p.freq = a->freq;
  p.x_sb = a->x_sb;
  p.x_st = a->x_sl;
  p.x_sh = a->x_sh;
  p.y_sb = a->y_sb;
  p.y_st = a->y_sl;
  p.y_sh = a->y_sh;
  p.pos_sb = a->pos_sb;
  p.pos64 = a->pos64;
  p.B = a->B;
  p.L = a->L;
  p.H = a->H;
  p.d = a->d;
  p.rot = a->rot;
  p.interleaved = a->interleaved ? 1 : 0;
  p.sign = a->inverse ? -1.0f : 1.0f;
  p.mscale = a->scale;
  const int vec = 16 / eb;
  const long long sx[3] = {a->x_sb, a->x_sl, a->x_sh}, sy[3] = {a->y_sb, a->y_sl, a->y_sh};
  const bool wide = rotary_vec(a->d, a->rot, p.interleaved, vec) &&
                    vector_ok(a->x, sx, 3, vec, eb) && vector_ok(a->y, sy, 3, vec, eb);
  const int places = blasst::rotary_places(a->d, a->rot, p.interleaved, wide ? vec : 1);
  // as many tokens per block as leave a thread one round of loads, while there
  // are blocks enough; few tokens: heads over blocks
  const int groups = std::max(1, 256 / std::min(places, 256));
  p.tb = 1;
  while (2 * p.tb <= groups && groups / (2 * p.tb) * blasst::kRotaryAhead >= a->H &&
         tokens >= 16ll * p.tb * sms)
    p.tb *= 2;
  const long long blocks = (tokens + p.tb - 1) / p.tb;
  if (blocks > 0x7fffffffll) return BLASST_EINVAL;
  p.hb = p.tb > 1 ? a->H : heads_per_block(blocks, a->H, places, sms);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((a->H + p.hb - 1) / p.hb));
  if (grid.y > 65535) return BLASST_EINVAL;
  const size_t smem = static_cast<size_t>(p.tb) * (a->rot / 2) * sizeof(float2);
  const cudaStream_t s = static_cast<cudaStream_t>(a->stream);
  if (a->dtype == BLASST_BF16)
    return wide ? launch_rotary<__nv_bfloat16, 8>(p, grid, smem, s)
                : launch_rotary<__nv_bfloat16, 1>(p, grid, smem, s);
  if (a->dtype == BLASST_FP16)
    return wide ? launch_rotary<__half, 8>(p, grid, smem, s)
                : launch_rotary<__half, 1>(p, grid, smem, s);
  return wide ? launch_rotary<float, 4>(p, grid, smem, s) : launch_rotary<float, 1>(p, grid, smem, s);
}

int blasst_append(const blasst_append_args* a) {
  // (without sequences there are no lengths and no table)
  if (!a || !a->k || !a->v || !a->k_pages || !a->v_pages || (a->n_seq > 0 && (!a->page_table || !a->kv_lens)) ||
      !a->cu_q || (a->q == nullptr) != (a->q_out == nullptr))
    return BLASST_EINVAL;
  if (a->dtype != BLASST_BF16 && a->dtype != BLASST_FP16 && a->dtype != BLASST_FP32)
    return BLASST_EUNSUPPORTED;
  if (a->n_seq < 0 || a->T < 0 || a->Hkv <= 0 || (a->q && a->Hq <= 0) || a->d <= 0 ||
      a->n_pages <= 0 || a->page_size <= 0 || a->table_width < 0 ||
      a->table_stride < a->table_width)
    return BLASST_EINVAL;
  if (a->freq ? (a->rot < 2 || a->rot > a->d || a->rot % 2 != 0) : a->rot != 0) return BLASST_EINVAL;
  if (a->freq && (!(a->scale > 0.0f) || !std::isfinite(a->scale))) return BLASST_EINVAL;
  if (a->d > 1024) return BLASST_EUNSUPPORTED;
  const int eb = elem_bytes(a->dtype);
  for (const void* ptr : {a->q, static_cast<const void*>(a->q_out), a->k, a->v,
                          static_cast<const void*>(a->k_pages), static_cast<const void*>(a->v_pages)})
    if (!aligned(ptr, eb)) return BLASST_EINVAL;
  if (!aligned(a->page_table, 4) || !aligned(a->kv_lens, 4) || !aligned(a->cu_q, 4) ||
      !aligned(a->freq, 8))
    return BLASST_EINVAL;
  if (a->q && a->q == a->q_out && (a->q_st != a->qo_st || a->q_sh != a->qo_sh)) return BLASST_EINVAL;
  if (a->T == 0 || a->n_seq == 0) return BLASST_OK;
  const int sms = sm_count();
  int* err = error_word();
  if (!err || sms == 0) return BLASST_ECUDA;
  blasst::AppendParams p{};
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.q_out = a->q_out;
  p.k_pages = a->k_pages;
  p.v_pages = a->v_pages;
  p.q_st = a->q_st;
  p.q_sh = a->q_sh;
  p.k_st = a->k_st;
  p.k_sh = a->k_sh;
  p.v_st = a->v_st;
  p.v_sh = a->v_sh;
  p.qo_st = a->qo_st;
  p.qo_sh = a->qo_sh;
  p.kp_sp = a->kp_sp;
  p.kp_st = a->kp_st;
  p.kp_sh = a->kp_sh;
  p.vp_sp = a->vp_sp;
  p.vp_st = a->vp_st;
  p.vp_sh = a->vp_sh;
  p.table = a->page_table;
  p.table_stride = a->table_stride;
  p.table_width = a->table_width;
  p.page_size = a->page_size;
  p.n_pages = a->n_pages;
  p.kv_lens = a->kv_lens;
  p.cu_q = a->cu_q;
  p.n_seq = a->n_seq;
  p.T = a->T;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.d = a->d;
  p.rot = a->rot;
  p.interleaved = a->interleaved ? 1 : 0;
  p.freq = a->freq;
  p.mscale = a->scale;
  p.err = err;
  const int vec = 16 / eb;
  const long long sq[4] = {a->q_st, a->q_sh, a->qo_st, a->qo_sh};
  const long long sk[5] = {a->k_st, a->k_sh, a->kp_sp, a->kp_st, a->kp_sh};
  const long long sv[5] = {a->v_st, a->v_sh, a->vp_sp, a->vp_st, a->vp_sh};
  bool wide = rotary_vec(a->d, a->rot, p.interleaved, vec) && vector_ok(a->k, sk, 5, vec, eb) &&
              vector_ok(a->k_pages, sk, 5, vec, eb) && vector_ok(a->v, sv, 5, vec, eb) &&
              vector_ok(a->v_pages, sv, 5, vec, eb);
  if (a->q) wide = wide && vector_ok(a->q, sq, 4, vec, eb) && vector_ok(a->q_out, sq, 4, vec, eb);
  const int places = blasst::rotary_places(a->d, a->rot, p.interleaved, wide ? vec : 1);
  const int heads = (a->q ? a->Hq : 0) + 2 * a->Hkv;
  const int groups = std::max(1, 256 / std::min(places, 256));
  p.tb = 1;
  while (2 * p.tb <= std::min(groups, blasst::kAppendTokens) && a->T >= 4ll * p.tb * sms) p.tb *= 2;
  const int blocks = (a->T + p.tb - 1) / p.tb;
  p.hb = p.tb > 1 ? heads : heads_per_block(blocks, heads, places, sms);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + p.hb - 1) / p.hb));
  if (grid.y > 65535) return BLASST_EINVAL;
  const size_t smem = static_cast<size_t>(p.tb) * std::max(1, a->rot / 2) * sizeof(float2);
  const cudaStream_t s = static_cast<cudaStream_t>(a->stream);
  if (a->dtype == BLASST_BF16)
    return wide ? launch_append<__nv_bfloat16, 8>(p, grid, smem, s)
                : launch_append<__nv_bfloat16, 1>(p, grid, smem, s);
  if (a->dtype == BLASST_FP16)
    return wide ? launch_append<__half, 8>(p, grid, smem, s)
                : launch_append<__half, 1>(p, grid, smem, s);
  return wide ? launch_append<float, 4>(p, grid, smem, s) : launch_append<float, 1>(p, grid, smem, s);
}

size_t blasst_seq_workspace_bytes(int d) {
  if (d != 64 && d != 128) return 0;
  return seq_workspace(sm_count(), d);
}

int blasst_packed_fwd(const blasst_packed_args* a) {
  // (a side without tokens has no pointers)
  if (!a || !a->q || (a->Tk > 0 && (!a->k || !a->v)) || !a->o || !a->lse || !a->cu_q || !a->cu_k)
    return BLASST_EINVAL;
  for (const void* ptr : {a->q, a->k, a->v, static_cast<const void*>(a->o),
                          static_cast<const void*>(a->lse)})
    if (!aligned(ptr, 16)) return BLASST_EINVAL;
  if (!aligned(a->cu_q, 4) || !aligned(a->cu_k, 4)) return BLASST_EINVAL;
  if (const int rc = check_heads(a->n_seq, a->Tq, a->Hq, a->Hkv, a->d, a->dtype)) return rc;
  if (a->Tk < 0 || std::isnan(a->scale)) return BLASST_EINVAL;
  for (long long st : {a->q_st, a->q_sh, a->k_st, a->k_sh, a->v_st, a->v_sh})
    if (!map_stride(st)) return BLASST_EINVAL;
  if (!aligned(a->workspace, 16) || !a->workspace) return BLASST_EWORKSPACE;
  if (a->n_seq == 0 || a->Tq == 0) return BLASST_OK;
  const int sms = sm_count();
  if (sms == 0) return BLASST_ECUDA;
  if (a->workspace_bytes < seq_workspace(sms, a->d)) return BLASST_EWORKSPACE;
  blasst::SeqAttnParams p{};
  p.err = error_word();
  if (!p.err) return BLASST_ECUDA;
  p.o = a->o;
  p.lse = a->lse;
  p.cu_q = a->cu_q;
  p.cu_k = a->cu_k;
  p.page_size = 1;
  p.n_pages = 1;
  p.chunk_log2 = 7;
  p.n_seq = a->n_seq;
  p.Tq = a->Tq;
  p.Tk = a->Tk;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.g = a->Hq / a->Hkv;
  p.causal = a->causal ? 1 : 0;
  // a map needs an address also where no tile is ever loaded
  const void* k = a->Tk > 0 ? a->k : a->q;
  const void* v = a->Tk > 0 ? a->v : a->q;
  CUtensorMap mk, mv;
  if (!make_map4(&mk, k, a->dtype, {a->d, a->Tk, a->Hkv, 1}, {a->k_st, a->k_sh, 8}, 128, 1) ||
      !make_map4(&mv, v, a->dtype, {a->d, a->Tk, a->Hkv, 1}, {a->v_st, a->v_sh, 8}, 128, 1))
    return BLASST_ECUDA;
  return run_seq(p, a->q, a->q_st, a->q_sh, a->d, a->scale, a->dtype, mk, mv, a->Tk, a->workspace, sms,
                 a->stream);
}

size_t blasst_packed_bwd_workspace_bytes(int Tq, int Hq, int Hkv) {
  if (Tq < 0 || Hq <= 0 || Hkv <= 0) return 0;
  return bwd_workspace(Tq, Hq, Hkv);
}

int blasst_packed_bwd(const blasst_packed_bwd_args* a) {
  if (!a || !a->cu_q || !a->cu_k) return BLASST_EINVAL;
  if (a->Tq > 0 && (!a->q || !a->o || !a->dout || !a->lse || !a->dq)) return BLASST_EINVAL;
  if (a->Tk > 0 && (!a->k || !a->v || !a->dk || !a->dv)) return BLASST_EINVAL;
  for (const void* ptr : {a->q, a->k, a->v, a->o, a->dout, static_cast<const void*>(a->lse),
                          static_cast<const void*>(a->dq), static_cast<const void*>(a->dk),
                          static_cast<const void*>(a->dv)})
    if (!aligned(ptr, 16)) return BLASST_EINVAL;
  if (!aligned(a->cu_q, 4) || !aligned(a->cu_k, 4)) return BLASST_EINVAL;
  if (const int rc = check_heads(a->n_seq, a->Tq, a->Hq, a->Hkv, a->d, a->dtype)) return rc;
  if (a->Tk < 0 || std::isnan(a->scale)) return BLASST_EINVAL;
  for (long long st : {a->q_st, a->q_sh, a->k_st, a->k_sh, a->v_st, a->v_sh, a->o_st, a->o_sh,
                       a->do_st, a->do_sh})
    if (!map_stride(st)) return BLASST_EINVAL;
  if (!aligned(a->workspace, 16) || !a->workspace ||
      a->workspace_bytes < bwd_workspace(a->Tq, a->Hq, a->Hkv))
    return BLASST_EWORKSPACE;
  if (a->n_seq == 0 || (a->Tq == 0 && a->Tk == 0)) return BLASST_OK;
  blasst::SeqBwdParams p{};
  p.g = a->Hq / a->Hkv;
  p.rt = 128 / p.g;
  // places for tiles (seq_place)
  const long long n_key = a->Tk > 0 ? a->Tk / 128 + static_cast<long long>(a->n_seq) : 0;
  const long long n_row = a->Tq > 0 ? a->Tq / p.rt + static_cast<long long>(a->n_seq) : 0;
  if ((n_key + n_row) * a->Hkv > 0x7fffffffll) return BLASST_EINVAL;
  p.n_key = static_cast<int>(n_key);
  p.n_row = static_cast<int>(n_row);
  p.err = error_word();
  if (!p.err) return BLASST_ECUDA;
  const bool f16 = a->dtype == BLASST_FP16;
  // bf16: pairs; fp16: the sizes of all rows, then D
  float2* stats = static_cast<float2*>(a->workspace);
  uint32_t* sizes = static_cast<uint32_t*>(a->workspace);
  float* dsum = reinterpret_cast<float*>(sizes + static_cast<size_t>(a->Tq) * a->Hq);
  p.dq = a->dq;
  p.dk = a->dk;
  p.dv = a->dv;
  p.stats = stats;
  p.dsum = dsum;
  p.sizes = sizes;
  p.lse = a->lse;
  p.k = a->k;
  p.k_st = a->k_st;
  p.k_sh = a->k_sh;
  p.cu_q = a->cu_q;
  p.cu_k = a->cu_k;
  p.n_seq = a->n_seq;
  p.Tq = a->Tq;
  p.Tk = a->Tk;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.causal = a->causal ? 1 : 0;
  const double sc = a->scale > 0.0f ? static_cast<double>(a->scale) : 1.0 / std::sqrt(static_cast<double>(a->d));
  p.scale = static_cast<float>(sc);
  p.scale_log2 = static_cast<float>(sc * 1.4426950408889634);
  p.timeout_ns = kTimeoutNs;
  blasst::SeqBwdRowsParams r{};
  r.o = a->o;
  r.dout = a->dout;
  r.v = a->v;
  r.lse = a->lse;
  r.stats = stats;
  r.dsum = dsum;
  r.sizes = sizes;
  r.cu_q = a->cu_q;
  r.cu_k = a->cu_k;
  r.o_st = a->o_st;
  r.o_sh = a->o_sh;
  r.do_st = a->do_st;
  r.do_sh = a->do_sh;
  r.v_st = a->v_st;
  r.v_sh = a->v_sh;
  r.n_seq = a->n_seq;
  r.Tq = a->Tq;
  r.Tk = a->Tk;
  r.Hq = a->Hq;
  r.Hkv = a->Hkv;
  r.g = p.g;
  r.row_blocks = static_cast<int>((static_cast<long long>(a->Tq) * p.g + blasst::kBwdRowsPerBlock - 1) /
                                  blasst::kBwdRowsPerBlock);
  // a map needs an address also where no tile is ever loaded
  const void* q = a->Tq > 0 ? a->q : a->k;
  const void* dout = a->Tq > 0 ? a->dout : a->k;
  const void* k = a->Tk > 0 ? a->k : a->q;
  const void* v = a->Tk > 0 ? a->v : a->q;
  CUtensorMap mq, mdo, mk, mv;
  if (!make_map4(&mq, q, a->dtype, {a->d, p.g, a->Tq, a->Hkv}, {a->q_sh, a->q_st, a->q_sh * p.g},
                 p.g, p.rt) ||
      !make_map4(&mdo, dout, a->dtype, {a->d, p.g, a->Tq, a->Hkv},
                 {a->do_sh, a->do_st, a->do_sh * p.g}, p.g, p.rt) ||
      !make_map4(&mk, k, a->dtype, {a->d, a->Tk, a->Hkv, 1}, {a->k_st, a->k_sh, 8}, 128, 1) ||
      !make_map4(&mv, v, a->dtype, {a->d, a->Tk, a->Hkv, 1}, {a->v_st, a->v_sh, 8}, 128, 1))
    return BLASST_ECUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(a->stream);
  if (!f16)
    return a->d == 128 ? launch_seq_bwd<128, __nv_bfloat16>(mq, mdo, mk, mv, p, r, s)
                       : launch_seq_bwd<64, __nv_bfloat16>(mq, mdo, mk, mv, p, r, s);
  return a->d == 128 ? launch_seq_bwd<128, __half>(mq, mdo, mk, mv, p, r, s)
                     : launch_seq_bwd<64, __half>(mq, mdo, mk, mv, p, r, s);
}

int blasst_paged_fwd(const blasst_paged_args* a) {
  // (without sequences there are no lengths and no table)
  if (!a || !a->q || !a->k_pages || !a->v_pages || !a->o || !a->lse || !a->cu_q ||
      (a->n_seq > 0 && (!a->page_table || !a->kv_lens)))
    return BLASST_EINVAL;
  for (const void* ptr : {a->q, a->k_pages, a->v_pages, static_cast<const void*>(a->o),
                          static_cast<const void*>(a->lse)})
    if (!aligned(ptr, 16)) return BLASST_EINVAL;
  if (!aligned(a->cu_q, 4) || !aligned(a->kv_lens, 4) || !aligned(a->page_table, 4)) return BLASST_EINVAL;
  if (const int rc = check_heads(a->n_seq, a->Tq, a->Hq, a->Hkv, a->d, a->dtype)) return rc;
  if (a->n_pages <= 0 || a->page_size <= 0 || a->table_width < 0 ||
      a->table_stride < a->table_width || std::isnan(a->scale))
    return BLASST_EINVAL;
  if (a->page_size % 8 != 0 || a->n_pages == 0x7fffffff) return BLASST_EUNSUPPORTED;
  for (long long st : {a->q_st, a->q_sh, a->kp_sp, a->kp_st, a->kp_sh, a->vp_sp, a->vp_st, a->vp_sh})
    if (!map_stride(st)) return BLASST_EINVAL;
  if (!aligned(a->workspace, 16) || !a->workspace) return BLASST_EWORKSPACE;
  if (a->n_seq == 0 || a->Tq == 0) return BLASST_OK;
  const int sms = sm_count();
  if (sms == 0) return BLASST_ECUDA;
  if (a->workspace_bytes < seq_workspace(sms, a->d)) return BLASST_EWORKSPACE;
  blasst::SeqAttnParams p{};
  p.err = error_word();
  if (!p.err) return BLASST_ECUDA;
  p.o = a->o;
  p.lse = a->lse;
  p.cu_q = a->cu_q;
  p.kv_lens = a->kv_lens;
  p.table = a->page_table;
  p.table_stride = a->table_stride;
  p.table_width = a->table_width;
  p.page_size = a->page_size;
  p.n_pages = a->n_pages;
  p.chunk_log2 = 3;
  while (p.chunk_log2 < 7 && a->page_size % (2 << p.chunk_log2) == 0) ++p.chunk_log2;
  p.n_seq = a->n_seq;
  p.Tq = a->Tq;
  p.Tk = 0;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.g = a->Hq / a->Hkv;
  p.causal = a->causal ? 1 : 0;
  CUtensorMap mk, mv;
  if (!make_map4(&mk, a->k_pages, a->dtype, {a->d, a->page_size, a->Hkv, a->n_pages},
                 {a->kp_st, a->kp_sh, a->kp_sp}, 1 << p.chunk_log2, 1) ||
      !make_map4(&mv, a->v_pages, a->dtype, {a->d, a->page_size, a->Hkv, a->n_pages},
                 {a->vp_st, a->vp_sh, a->vp_sp}, 1 << p.chunk_log2, 1))
    return BLASST_ECUDA;
  return run_seq(p, a->q, a->q_st, a->q_sh, a->d, a->scale, a->dtype, mk, mv,
                 static_cast<long long>(a->table_width) * a->page_size, a->workspace, sms, a->stream);
}

}  // extern "C"
