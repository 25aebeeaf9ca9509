// moe_paged_attention and moe_tree_attention: checks, workspace and launch (the kernels are in attn.cuh).
#include <cudaTypedefs.h>

#include "attn.cuh"

struct moe_attn_ws {
  int Hq, Hkv, D, sms, phantom;
  int32_t* error;
  float *part, *ml;
  int4* join;
};

namespace moe {
namespace attn {
int launch_d64(const Args& a, int e4m3, int nr, int sms, cudaStream_t s);
int launch_d128(const Args& a, int e4m3, int nr, int sms, cudaStream_t s);
int launch_d256(const Args& a, int e4m3, int nr, int sms, cudaStream_t s);
int launch_tree_d64(const Args& a, int e4m3, int nr, int sms, cudaStream_t s);
int launch_tree_d128(const Args& a, int e4m3, int nr, int sms, cudaStream_t s);
int launch_tree_d256(const Args& a, int e4m3, int nr, int sms, cudaStream_t s);
int opt_in_tree_d64();
int opt_in_tree_d128();
int opt_in_tree_d256();
int opt_in_d64();
int opt_in_d128();
int opt_in_d256();

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// Tiles of a pool or of the query rows; what lies outside reads as zeros.
bool encode(CUtensorMap* m, void* base, int e4m3, int rank, const cuuint64_t* dims, const cuuint64_t* pitches,
            const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  return fn && fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, base, dims, pitches,
                  box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace attn
}  // namespace moe

extern "C" int moe_attn_ws_create(moe_attn_ws** out, int Hq, int Hkv, int D) {
  using namespace moe;
  if (!out || Hkv < 1 || Hkv > 1024 || Hq < 1 || Hq % Hkv || Hq / Hkv > kMaxGroup || (D != 64 && D != 128 && D != 256))
    return MOE_EINVAL;
  *out = nullptr;
  moe_attn_ws* w = static_cast<moe_attn_ws*>(calloc(1, sizeof(moe_attn_ws)));
  if (!w) return MOE_ENOMEM;
  w->Hq = Hq;
  w->Hkv = Hkv;
  w->D = D;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1 ||
      (D == 64 ? attn::opt_in_d64() : D == 128 ? attn::opt_in_d128() : attn::opt_in_d256()) != MOE_OK ||
      (D == 64 ? attn::opt_in_tree_d64() : D == 128 ? attn::opt_in_tree_d128() : attn::opt_in_tree_d256()) != MOE_OK) {
    cudaGetLastError();
    free(w);
    return MOE_ECUDA;
  }
  w->sms = sms;
  const size_t runs = 2 * size_t(sms);
  const size_t rows = 2 * runs * (D == 256 ? 64 : attn::kChunkRows);
  const size_t o_part = 256, o_ml = o_part + rows * D * 4, o_join = o_ml + rows * 8;
  const size_t bytes = o_join + runs * 16;
  uint8_t* base = nullptr;
  if (cudaMalloc(&base, bytes) != cudaSuccess) {
    cudaGetLastError();
    free(w);
    return MOE_ENOMEM;
  }
  w->error = reinterpret_cast<int32_t*>(base);
  w->part = reinterpret_cast<float*>(base + o_part);
  w->ml = reinterpret_cast<float*>(base + o_ml);
  w->join = reinterpret_cast<int4*>(base + o_join);
  if (cudaMemset(base, 0, bytes) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    moe_attn_ws_destroy(w);
    return MOE_ECUDA;
  }
  *out = w;
  return MOE_OK;
}

extern "C" int moe_attn_ws_destroy(moe_attn_ws* w) {
  if (!w) return MOE_OK;
  cudaFree(w->error);  // the start of the single allocation
  free(w);
  return MOE_OK;
}

extern "C" int moe_attn_ws_get_view(const moe_attn_ws* w, moe_attn_ws_view* v) {
  if (!w || !v) return MOE_EINVAL;
  v->error = w->error;
  return MOE_OK;
}

extern "C" int moe_attn_ws_set_wait_test(moe_attn_ws* w, int stage) {
  if (!w || stage < 0 || stage > 3) return MOE_EINVAL;
  w->phantom = stage;
  return MOE_OK;
}

extern "C" int moe_attn_sync_status(moe_attn_ws* w, moe_stream_t stream) {
  if (!w) return MOE_EINVAL;
  // all on the caller's stream: a reset elsewhere could run after the stream's next call has recorded its error
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int32_t e = 0;
  MOE_CUDA_TRY(cudaMemcpyAsync(&e, w->error, 4, cudaMemcpyDeviceToHost, s));
  MOE_CUDA_TRY(cudaMemsetAsync(w->error, 0, 4, s));
  MOE_CUDA_TRY(cudaStreamSynchronize(s));
  return e;
}

namespace moe {
namespace {
// Both calls; tree null: a request's new tokens follow one another.
int attend(const moe_kv_pages* kv, const moe_kv_batch* b, const moe_tree* tree, const uint16_t* q, long long q_stride, int Hq,
           uint16_t* o, long long o_stride, float scale, int window, moe_attn_ws* ws, moe_stream_t stream) {
  attn::Args a = {};
  const int rc = kv_view(kv, b, &a.kv);
  if (rc) return rc;
  if (!ws || Hq != ws->Hq || kv->Hkv != ws->Hkv || kv->D != ws->D || window < 0 || !isfinite(scale)) return MOE_EINVAL;
  const int T = b->T;
  if (T == 0 || b->B == 0) return MOE_OK;
  const long long width = (long long)Hq * kv->D;
  if (!rows_ok(q, q_stride, T, width) || !rows_ok(o, o_stride, T, width)) return MOE_EINVAL;
  const int G = Hq / kv->Hkv, n = b->max_n > 1 ? b->max_n : 1;
  const int nr = tree ? attn::tree_row_tile(kv->D, G, n, kv->e4m3) : attn::row_tile(kv->D, G, n);
  a.o = o;
  a.os = T > 1 ? o_stride : width;
  a.q = q;
  a.qs = T > 1 ? q_stride : width;
  a.G = G;
  a.window = window < attn::cap_of(a.kv) ? window : 0;  // one that holds every key is none
  const int tile = nr == attn::kChunkRows ? nr / 2 / a.G : nr / a.G;  // tokens of a row tile
  a.tokens = nr == attn::kChunkRows ? 2 * tile : tile;
  // the schedule counts in 31 bits: a unit has at most its request's tiles, and three more places, of a tree six
  const int more = tree ? 7 : 4;
  if ((double(T) / a.tokens + b->B) * kv->Hkv * (double(a.kv.table_stride) * kv->page / attn::kKeys + more) > 2147483000.0)
    return MOE_EINVAL;
  const int size = kv->e4m3 ? 1 : 2, box = kv->page < attn::kKeys ? kv->page : attn::kKeys;
  // sizes and byte strides of the pools, innermost first; a size of one takes any stride
  const cuuint64_t dims[4] = {cuuint64_t(kv->D), cuuint64_t(kv->page), cuuint64_t(kv->Hkv), cuuint64_t(kv->npages)};
  auto pitch = [&](long long bytes) { return cuuint64_t(bytes ? bytes : kv->D * size); };
  const cuuint64_t pitches[3] = {pitch(a.kv.tok_stride), pitch(a.kv.head_stride), pitch(a.kv.page_stride)};
  const cuuint32_t boxes[4] = {cuuint32_t(kv->e4m3 ? (kv->D < 128 ? kv->D : 128) : 64), cuuint32_t(box), 1, 1};
  const cuuint64_t qdims[3] = {cuuint64_t(kv->D), cuuint64_t(Hq), cuuint64_t(T)};
  const cuuint64_t qpitches[2] = {cuuint64_t(kv->D) * 2, cuuint64_t(T > 1 ? q_stride : width) * 2};
  const cuuint32_t qbox[3] = {64, cuuint32_t(a.G), cuuint32_t(tile)};
  // operands of the tensor core are swizzled by their rows; E4M3 values, and a chunk's keys, become one later
  const CUtensorMapSwizzle k_swizzle = !kv->e4m3 ? CU_TENSOR_MAP_SWIZZLE_128B
                                       : nr >= attn::kWideRows ? CU_TENSOR_MAP_SWIZZLE_NONE
                                       : kv->D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  const CUtensorMapSwizzle v_swizzle = kv->e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
  if (!attn::encode(&a.mk, kv->k, kv->e4m3, 4, dims, pitches, boxes, k_swizzle) ||
      !attn::encode(&a.mv, kv->v, kv->e4m3, 4, dims, pitches, boxes, v_swizzle) ||
      !attn::encode(&a.mq, const_cast<uint16_t*>(q), 0, 3, qdims, qpitches, qbox, CU_TENSOR_MAP_SWIZZLE_128B))
    return MOE_EINVAL;
  if (tree) {
    a.above = tree->above;
    a.below = tree->below;
    a.depth = tree->depth;
    a.words = tree->words;
  }
  a.scale = scale;
  a.phantom = ws->phantom;
  a.err = ws->error;
  a.part = ws->part;
  a.ml = ws->ml;
  a.join = ws->join;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (kv->D) {
    case 64: return (tree ? attn::launch_tree_d64 : attn::launch_d64)(a, kv->e4m3, nr, ws->sms, s);
    case 128: return (tree ? attn::launch_tree_d128 : attn::launch_d128)(a, kv->e4m3, nr, ws->sms, s);
    default: return (tree ? attn::launch_tree_d256 : attn::launch_d256)(a, kv->e4m3, nr, ws->sms, s);
  }
}
}  // namespace
}  // namespace moe

extern "C" int moe_paged_attention(const moe_kv_pages* kv, const moe_kv_batch* b, const uint16_t* q, long long q_stride,
                                   int Hq, uint16_t* o, long long o_stride, float scale, int window, moe_attn_ws* ws,
                                   moe_stream_t stream) {
  return moe::attend(kv, b, nullptr, q, q_stride, Hq, o, o_stride, scale, window, ws, stream);
}

extern "C" int moe_tree_attention(const moe_kv_pages* kv, const moe_kv_batch* b, const moe_tree* tree, const uint16_t* q,
                                  long long q_stride, int Hq, uint16_t* o, long long o_stride, float scale, int window,
                                  moe_attn_ws* ws, moe_stream_t stream) {
  if (!b || !tree || tree->words < 1 || tree->words > 8) return MOE_EINVAL;
  if (b->B > 0 && b->T > 0 && (!tree->above || !tree->below || !tree->depth)) return MOE_EINVAL;
  return moe::attend(kv, b, tree, q, q_stride, Hq, o, o_stride, scale, window, ws, stream);
}
