// attn_api.cu -- the C ABI declared in include/attn.h: argument validation,
// tensor-map encoding, backward scratch, launch bookkeeping and the sticky
// device status word.  Every step of the computation runs in the kernels of
// attn_fwd.cu / attn_bwd.cu; this file only checks and marshals.
#include <cmath>
#include <cstdint>
#include <atomic>
#include <initializer_list>
#include <cstring>
#include <mutex>

#include "attn.h"
#include "attn_internal.h"
#include "attn_paged.h"

// Sticky device-side status (one copy per device that loads the library).
__device__ int g_attn_status;
// Sticky word of the paged kernels' checks of tables and lengths.  Apart from
// g_attn_status, which a pipeline wait reads to stop early: a bad table entry
// must not stop an unrelated call.
__device__ int g_attn_check;

namespace attn {
namespace {

constexpr int kMaxDevices = 64;
thread_local int t_last_launches = 0;

std::mutex g_mu;
int* g_status_ptr[kMaxDevices] = {};
int* g_check_ptr[kMaxDevices] = {};
int g_arch_ok[kMaxDevices] = {};  // 0 unknown, 1 ok, -1 wrong arch
cuuint64_t g_smem_attr_done[kMaxDevices][8] = {};
const void* g_smem_attr_func[kMaxDevices][8] = {};

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// Current device, checked to be compute capability 10.3; returns a status.
int current_device(int* dev) {
  if (cudaGetDevice(dev) != cudaSuccess) return kStatusCuda;
  if (*dev < 0 || *dev >= kMaxDevices) return kStatusUnsupported;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_arch_ok[*dev] == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev) != cudaSuccess)
      return kStatusCuda;
    g_arch_ok[*dev] = (major == 10 && minor == 3) ? 1 : -1;
  }
  return g_arch_ok[*dev] == 1 ? kStatusOk : kStatusArch;
}

int* status_ptr(int dev) {
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_status_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_attn_status) != cudaSuccess) return nullptr;
    g_status_ptr[dev] = static_cast<int*>(p);
  }
  return g_status_ptr[dev];
}

int* check_ptr(int dev) {
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_check_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_attn_check) != cudaSuccess) return nullptr;
    g_check_ptr[dev] = static_cast<int*>(p);
  }
  return g_check_ptr[dev];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Checks shared by forward and backward.  Pure host logic: no CUDA call.
int validate_common(int B, int H, int N, int d, float scale) {
  if (B < 1 || H < 1 || N < 1) return kStatusInvalid;
  if (!std::isfinite(scale)) return kStatusInvalid;
  if (d != 32 && d != 64 && d != 128) return kStatusUnsupported;
  const int64_t BH = static_cast<int64_t>(B) * H;
  if (BH > 65535) return kStatusUnsupported;           // grid.y limit
  if (N > (1 << 24)) return kStatusUnsupported;         // keeps row indices and TMA coords in range
  return kStatusOk;
}

}  // namespace

bool encode_bhnd_map(CUtensorMap* map, const void* base, int BH, int N, int d, int box_inner,
                     int box_rows, int row_bytes, bool bf16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                              static_cast<cuuint64_t>(BH)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                                 static_cast<cuuint64_t>(N) * static_cast<cuuint64_t>(d) * 2};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows),
                             1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapSwizzle swz =
      row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_map_u8(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                   uint64_t stride1, uint64_t stride2, uint32_t b0, uint32_t b1) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {stride1, stride2};
  const cuuint32_t box[3] = {b0, b1, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_pages_map(CUtensorMap* map, const void* base, int row, int page, int heads, int pages, int64_t tok,
                      int64_t head, int64_t page_stride, int box_bytes, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(page),
                              static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(tok), static_cast<cuuint64_t>(head),
                                 static_cast<cuuint64_t>(page_stride)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(box_bytes), static_cast<cuuint32_t>(box_rows), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle swz = box_bytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                 : box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                   : CU_TENSOR_MAP_SWIZZLE_32B;
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool ensure_smem_attr(const void* func, int bytes) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  std::lock_guard<std::mutex> lk(g_mu);
  for (int i = 0; i < 8; ++i) {
    if (g_smem_attr_func[dev][i] == func && g_smem_attr_done[dev][i] >= (cuuint64_t)bytes) return true;
  }
  if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return false;
  for (int i = 0; i < 8; ++i) {
    if (g_smem_attr_func[dev][i] == nullptr || g_smem_attr_func[dev][i] == func) {
      g_smem_attr_func[dev][i] = func;
      g_smem_attr_done[dev][i] = static_cast<cuuint64_t>(bytes);
      break;
    }
  }
  return true;
}

bool check_launch_regs(const void* func, int regs) {
  // The register count is a property of the compiled kernel: look it up once
  // per kernel (cudaFuncGetAttributes costs about a microsecond per call).
  static std::mutex mu;
  static const void* seen_func[64] = {};
  static int seen_regs[64] = {};
  {
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < 64 && seen_func[i]; ++i)
      if (seen_func[i] == func) return seen_regs[i] == regs;
  }
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, func) != cudaSuccess) return false;
  std::lock_guard<std::mutex> lk(mu);
  for (int i = 0; i < 64; ++i) {
    if (seen_func[i] == func) break;
    if (!seen_func[i]) {
      seen_func[i] = func;
      seen_regs[i] = fa.numRegs;
      break;
    }
  }
  return fa.numRegs == regs;
}

int device_sm_count() {
  static std::atomic<int> count[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int n = count[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 0;
  count[dev].store(n, std::memory_order_relaxed);
  return n;
}

int bwd_tail_split(int BH, int N, int causal) {
  return bwd_tail_split_items(BH, N, causal, device_sm_count());
}

int* status_word_current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  return status_ptr(dev);
}

BwdScratch bwd_scratch_layout(int BH, int N, int d) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t Npad = static_cast<size_t>((N + 127) / 128) * 128;
  BwdScratch s;
  s.dq_off = 0;
  s.lse2_off = up(static_cast<size_t>(BH) * N * d * sizeof(float));
  s.d_off = s.lse2_off + up(static_cast<size_t>(BH) * Npad * sizeof(float));
  s.total = s.d_off + up(static_cast<size_t>(BH) * Npad * sizeof(float));
  return s;
}

namespace {

constexpr DropParams kNoDrop = {0u, 0u, 0u, 0u, 1.f};

// Dropout probability -> keep threshold and Philox key.  t = 256 keeps
// everything, which is no dropout (t = 0 in the result).
int make_drop(float p, unsigned long long seed, unsigned int offset, DropParams* out) {
  if (!std::isfinite(p) || p < 0.f || p >= 1.f) return kStatusInvalid;
  const double t = std::floor((1.0 - static_cast<double>(p)) * 256.0 + 0.5);
  if (t < 1.0) return kStatusInvalid;
  *out = kNoDrop;
  if (t >= 256.0) return kStatusOk;
  out->t = static_cast<uint32_t>(t);
  out->k0 = static_cast<uint32_t>(seed);
  out->k1 = static_cast<uint32_t>(seed >> 32);
  out->offset = offset;
  out->rscale = static_cast<float>(256.0 / t);
  return kStatusOk;
}

int fwd_entry(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
              int N, int d, float scale, int causal, void* stream, bool bf16,
              const DropParams& drop = kNoDrop) {
  if (!q || !k || !v || !o || !lse) return kStatusInvalid;
  int rc = validate_common(B, H, N, d, scale);
  if (rc) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return kStatusInvalid;
  const size_t nbytes = static_cast<size_t>(B) * H * N * d * 2;
  const size_t lbytes = static_cast<size_t>(B) * H * N * 4;
  for (const void* in : {q, k, v})
    if (overlaps(o, nbytes, in, nbytes) || overlaps(lse, lbytes, in, nbytes)) return kStatusInvalid;
  if (overlaps(o, nbytes, lse, lbytes)) return kStatusInvalid;
  int dev = 0;
  if ((rc = current_device(&dev))) return rc;
  int* st = status_ptr(dev);
  if (!st) return kStatusCuda;
  FwdArgs a;
  a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
  a.BH = B * H; a.N = N; a.d = d;
  a.sl2 = std::fabs(scale) * 1.4426950408889634f;
  a.causal = causal ? 1 : 0;
  a.negate = scale < 0.f ? 1 : 0;
  a.bf16 = bf16;
  a.stream = static_cast<cudaStream_t>(stream);
  a.status = st;
  a.drop = drop;
  rc = launch_fwd(a);
  if (rc == kStatusOk) t_last_launches = 1;
  return rc;
}

int bwd_entry(const void* q, const void* k, const void* v, const void* o, const void* dO,
              const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
              float scale, int causal, void* stream, bool bf16, const DropParams& drop = kNoDrop,
              const uint8_t* bmask = nullptr, int mask_heads = 1) {
  if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return kStatusInvalid;
  int rc = validate_common(B, H, N, d, scale);
  if (rc) return rc;
  for (const void* p : {q, k, v, o, dO, static_cast<const void*>(dq), static_cast<const void*>(dk),
                        static_cast<const void*>(dv)})
    if (!aligned16(p)) return kStatusInvalid;
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return kStatusInvalid;
  const size_t nbytes = static_cast<size_t>(B) * H * N * d * 2;
  const size_t lbytes = static_cast<size_t>(B) * H * N * 4;
  for (const void* out : {static_cast<const void*>(dq), static_cast<const void*>(dk),
                          static_cast<const void*>(dv)}) {
    for (const void* in : {q, k, v, o, dO})
      if (overlaps(out, nbytes, in, nbytes)) return kStatusInvalid;
    if (overlaps(out, nbytes, lse, lbytes)) return kStatusInvalid;
  }
  if (overlaps(dq, nbytes, dk, nbytes) || overlaps(dq, nbytes, dv, nbytes) ||
      overlaps(dk, nbytes, dv, nbytes))
    return kStatusInvalid;
  int dev = 0;
  if ((rc = current_device(&dev))) return rc;
  int* st = status_ptr(dev);
  if (!st) return kStatusCuda;
  const BwdScratch lay = bwd_scratch_layout(B * H, N, d);
  const int tail = bmask ? 0 : bwd_tail_split(B * H, N, causal);
  const size_t part_bytes = static_cast<size_t>(tail) * 4 * 128 * d * sizeof(float);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* ws = nullptr;
  if (cudaMallocAsync(&ws, lay.total + part_bytes, s) != cudaSuccess) return kStatusCuda;
  BwdArgs a;
  a.q = q; a.k = k; a.v = v; a.o = o; a.dO = dO; a.lse = lse;
  a.dq = dq; a.dk = dk; a.dv = dv;
  a.BH = B * H; a.N = N; a.d = d;
  a.sl2 = std::fabs(scale) * 1.4426950408889634f;
  a.scale = scale;
  a.causal = causal ? 1 : 0;
  a.negate = scale < 0.f ? 1 : 0;
  a.bf16 = bf16;
  a.stream = s;
  a.status = st;
  a.ws_dq = reinterpret_cast<float*>(static_cast<char*>(ws) + lay.dq_off);
  a.ws_lse2 = reinterpret_cast<float*>(static_cast<char*>(ws) + lay.lse2_off);
  a.ws_d = reinterpret_cast<float*>(static_cast<char*>(ws) + lay.d_off);
  a.drop = drop;
  a.bmask = bmask;
  a.H = H;
  a.mask_heads = mask_heads;
  a.tail_split = tail;
  a.ws_part = tail ? reinterpret_cast<float*>(static_cast<char*>(ws) + lay.total) : nullptr;
  rc = launch_bwd(a);
  const cudaError_t fe = cudaFreeAsync(ws, s);
  if (rc == kStatusOk && fe != cudaSuccess) rc = kStatusCuda;
  if (rc == kStatusOk) t_last_launches = 3;
  return rc;
}

int blocksparse_entry(const void* q, const void* k, const void* v, void* o, float* lse,
                      const uint8_t* mask, int mask_heads, int B, int H, int N, int d, float scale,
                      int causal, void* stream, bool bf16, const DropParams& drop = kNoDrop) {
  if (!mask) return kStatusInvalid;
  if (mask_heads != 1 && mask_heads != H) return kStatusInvalid;
  if ((N + 127) / 128 > kMaxSparseTiles) return kStatusUnsupported;
  if (!q || !k || !v || !o || !lse) return kStatusInvalid;
  int rc = validate_common(B, H, N, d, scale);
  if (rc) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return kStatusInvalid;
  const size_t nbytes = static_cast<size_t>(B) * H * N * d * 2;
  const size_t lbytes = static_cast<size_t>(B) * H * N * 4;
  for (const void* in : {q, k, v})
    if (overlaps(o, nbytes, in, nbytes) || overlaps(lse, lbytes, in, nbytes)) return kStatusInvalid;
  if (overlaps(o, nbytes, lse, lbytes)) return kStatusInvalid;
  int dev = 0;
  if ((rc = current_device(&dev))) return rc;
  int* st = status_ptr(dev);
  if (!st) return kStatusCuda;
  FwdArgs a;
  a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
  a.BH = B * H; a.N = N; a.d = d;
  a.sl2 = std::fabs(scale) * 1.4426950408889634f;
  a.causal = causal ? 1 : 0;
  a.negate = scale < 0.f ? 1 : 0;
  a.bf16 = bf16;
  a.stream = static_cast<cudaStream_t>(stream);
  a.status = st;
  a.bmask = mask;
  a.H = H;
  a.mask_heads = mask_heads;
  a.drop = drop;
  rc = launch_fwd(a);
  if (rc == kStatusOk) t_last_launches = 1;
  return rc;
}

int decode_entry(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                 int L, int d, float scale, void* stream) {
  if (!q || !k || !v || !o || !lse) return kStatusInvalid;
  int rc = validate_common(B, H, L, d, scale);
  if (rc) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return kStatusInvalid;
  const size_t qbytes = static_cast<size_t>(B) * H * d * 2;
  const size_t kvbytes = qbytes * static_cast<size_t>(L);
  const size_t lbytes = static_cast<size_t>(B) * H * 4;
  for (const void* in : {q, k, v}) {
    const size_t n = in == q ? qbytes : kvbytes;
    if (overlaps(o, qbytes, in, n) || overlaps(lse, lbytes, in, n)) return kStatusInvalid;
  }
  if (overlaps(o, qbytes, lse, lbytes)) return kStatusInvalid;
  int dev = 0;
  if ((rc = current_device(&dev))) return rc;
  DecodeArgs a;
  a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
  a.BH = B * H; a.L = L; a.d = d;
  a.sl2 = scale * 1.4426950408889634f;
  a.splits = decode_splits(a.BH, L);
  a.stream = static_cast<cudaStream_t>(stream);
  const size_t ws_bytes = static_cast<size_t>(a.BH) * a.splits * (d + 2) * sizeof(float);
  void* ws = nullptr;
  if (cudaMallocAsync(&ws, ws_bytes, a.stream) != cudaSuccess) return kStatusCuda;
  a.ws = static_cast<float*>(ws);
  rc = launch_decode(a);
  const cudaError_t fe = cudaFreeAsync(ws, a.stream);
  if (rc == kStatusOk && fe != cudaSuccess) rc = kStatusCuda;
  if (rc == kStatusOk) t_last_launches = 2;
  return rc;
}

int fp8_entry(const void* q, const void* k, const void* v, float dq_s, float dk_s, float dv_s, void* o,
              float* lse, int B, int H, int N, int d, float scale, int causal, void* stream) {
  if (!q || !k || !v || !o || !lse) return kStatusInvalid;
  int rc = validate_common(B, H, N, d, scale);
  if (rc) return rc;
  if (!std::isfinite(dq_s) || !std::isfinite(dk_s) || !std::isfinite(dv_s) || dq_s <= 0.f ||
      dk_s <= 0.f || dv_s <= 0.f)
    return kStatusInvalid;
  if (d != 128 || scale < 0.f) return kStatusUnsupported;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return kStatusInvalid;
  const size_t ibytes = static_cast<size_t>(B) * H * N * d;  // one byte per input element
  const size_t obytes = ibytes * 2, lbytes = static_cast<size_t>(B) * H * N * 4;
  for (const void* in : {q, k, v})
    if (overlaps(o, obytes, in, ibytes) || overlaps(lse, lbytes, in, ibytes)) return kStatusInvalid;
  if (overlaps(o, obytes, lse, lbytes)) return kStatusInvalid;
  int dev = 0;
  if ((rc = current_device(&dev))) return rc;
  int* st = status_ptr(dev);
  if (!st) return kStatusCuda;
  Fp8Args a;
  a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
  a.BH = B * H; a.N = N; a.d = d;
  a.sl2 = scale * dq_s * dk_s * 1.4426950408889634f;
  a.descale_v = dv_s;
  a.causal = causal ? 1 : 0;
  a.stream = static_cast<cudaStream_t>(stream);
  a.status = st;
  const size_t Npad = static_cast<size_t>((N + 127) / 128) * 128;
  void* ws = nullptr;
  if (cudaMallocAsync(&ws, static_cast<size_t>(a.BH) * 128 * Npad, a.stream) != cudaSuccess)
    return kStatusCuda;
  a.ws_vt = static_cast<uint8_t*>(ws);
  rc = launch_fwd_fp8(a);
  const cudaError_t fe = cudaFreeAsync(ws, a.stream);
  if (rc == kStatusOk && fe != cudaSuccess) rc = kStatusCuda;
  if (rc == kStatusOk) t_last_launches = 2;
  return rc;
}

}  // namespace
}  // namespace attn

namespace attn {
namespace {

// ---------------------------------------------------------------- paged cache

struct Dim {
  int64_t n, stride;  // extent, stride in bytes
};

// Strides of a tensor whose rows hold `row` contiguous bytes: multiples of 16;
// for outputs also such that no two rows share a byte (each stride, in
// ascending order, steps over all that the smaller ones span).
bool strides_ok(Dim* dims, int count, int64_t row, bool output) {
  for (int i = 0; i < count; ++i) {
    if (dims[i].n == 1) dims[i].stride = row;  // never stepped along
    if (dims[i].stride < 0 || dims[i].stride % 16 || dims[i].stride >= (int64_t{1} << 40)) return false;
  }
  if (!output) return true;
  Dim s[3];
  std::copy(dims, dims + count, s);
  std::sort(s, s + count, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
  int64_t span = row;
  for (int i = 0; i < count; ++i) {
    if (s[i].n == 1) continue;
    if (s[i].stride < span) return false;
    span = s[i].stride * (s[i].n - 1) + span;
  }
  return true;
}

size_t span_of(const Dim* dims, int count, int64_t row) {
  int64_t n = row;
  for (int i = 0; i < count; ++i) n += (dims[i].n - 1) * dims[i].stride;
  return static_cast<size_t>(n);
}

struct Span {
  const void* p;
  size_t n;
};

bool any_overlap(const Span& out, std::initializer_list<Span> others) {
  for (const Span& o : others)
    if (o.p && out.p && overlaps(out.p, out.n, o.p, o.n)) return true;
  return false;
}

// What the calls and the workspace queries take of a cache's sizes.
int paged_sizes(const attn_paged_kv_t* c) {
  if (c->B < 1 || c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->max_pages < 1) return kStatusInvalid;
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return kStatusUnsupported;
  if (c->page_size % 8 || c->page_size > 1024) return kStatusUnsupported;
  // B is a grid's y; (sequence, head) pairs are counted in x and in 64 bits only.
  if (c->B > 65535 || c->kv_heads > 65535 || static_cast<int64_t>(c->B) * c->kv_heads > (c->B <= 8192 ? 1 << 20 : 65535))
    return kStatusUnsupported;
  if (static_cast<int64_t>(c->max_pages) * c->page_size > (int64_t{1} << 30)) return kStatusUnsupported;
  return kStatusOk;
}

int query_heads_ok(int q_heads, int B, int H) {
  if (q_heads < 1 || q_heads % H) return kStatusInvalid;
  // No grid has a block to every (sequence, query head); a row of o's heads counts in int.
  if (q_heads > 65535) return kStatusUnsupported;
  return q_heads / H > 1024 && static_cast<int64_t>(B) * q_heads > 65535 ? kStatusUnsupported : kStatusOk;
}

bool listed_pages_ok(int n, int page) { return n >= 1 && static_cast<int64_t>(n) * page <= (int64_t{1} << 30); }

// What the library needs of a cache, in bytes; host logic only.
int paged_kv(const attn_paged_kv_t* c, int x_type, PagedKv* kv, Span* ks, Span* vs) {
  if (!c || !c->k_pages || !c->v_pages || !c->block_table || !c->seq_lens) return kStatusInvalid;
  if (const int rc = paged_sizes(c)) return rc;
  if (c->type != kTypeBf16 && c->type != kTypeF16 && c->type != kTypeE4m3) return kStatusInvalid;
  if (x_type != kTypeBf16 && x_type != kTypeF16) return kStatusInvalid;
  if (c->type != kTypeE4m3 && c->type != x_type) return kStatusInvalid;
  if (!std::isfinite(c->k_scale) || !std::isfinite(c->v_scale) || c->k_scale <= 0.f || c->v_scale <= 0.f)
    return kStatusInvalid;
  if (c->type != kTypeE4m3 && (c->k_scale != 1.f || c->v_scale != 1.f)) return kStatusInvalid;
  if (c->table_stride < 0 || (c->B > 1 && c->table_stride < c->max_pages)) return kStatusInvalid;
  if ((c->k_min == nullptr) != (c->k_max == nullptr)) return kStatusInvalid;
  for (const void* p : {static_cast<const void*>(c->k_pages), static_cast<const void*>(c->v_pages),
                        static_cast<const void*>(c->k_min), static_cast<const void*>(c->k_max)})
    if (!aligned16(p)) return kStatusInvalid;
  if ((reinterpret_cast<uintptr_t>(c->block_table) & 3u) || (reinterpret_cast<uintptr_t>(c->seq_lens) & 3u))
    return kStatusInvalid;
  const int e = type_bytes(c->type);
  const int64_t row = static_cast<int64_t>(c->head_dim) * e;
  for (int which = 0; which < 2; ++which) {
    const long long* st = which ? c->v_strides : c->k_strides;
    for (int i = 0; i < 3; ++i)
      if (st[i] < 0 || st[i] >= (1ll << 40)) return kStatusInvalid;
    Dim dims[3] = {{c->num_pages, st[0] * e}, {c->kv_heads, st[1] * e}, {c->page_size, st[2] * e}};
    if (!strides_ok(dims, 3, row, true)) return kStatusInvalid;
    *(which ? vs : ks) = {which ? c->v_pages : c->k_pages, span_of(dims, 3, row)};
    (which ? kv->v_page : kv->k_page) = dims[0].stride;
    (which ? kv->v_head : kv->k_head) = dims[1].stride;
    (which ? kv->v_tok : kv->k_tok) = dims[2].stride;
  }
  if (c->k_pages == c->v_pages) return kStatusInvalid;
  const size_t sum = static_cast<size_t>(c->num_pages) * c->kv_heads * row;
  if (c->k_min && (overlaps(c->k_min, sum, c->k_max, sum) || any_overlap({c->k_min, sum}, {*ks, *vs}) ||
                   any_overlap({c->k_max, sum}, {*ks, *vs})))
    return kStatusInvalid;
  kv->k = static_cast<uint8_t*>(c->k_pages);
  kv->v = static_cast<uint8_t*>(c->v_pages);
  kv->kmin = static_cast<uint8_t*>(c->k_min);
  kv->kmax = static_cast<uint8_t*>(c->k_max);
  kv->table = c->block_table;
  kv->table_stride = c->table_stride;
  kv->lens = c->seq_lens;
  kv->num_pages = c->num_pages;
  kv->page = c->page_size;
  kv->H = c->kv_heads;
  kv->d = c->head_dim;
  kv->max_pages = c->max_pages;
  kv->B = c->B;
  kv->type = c->type;
  kv->k_scale = c->k_scale;
  kv->v_scale = c->v_scale;
  return kStatusOk;
}

// Rows [rows][heads][d] of two-byte elements.
int paged_rows(const attn_rows_t* r, int64_t rows, int heads, int d, bool output, PagedRows* out, Span* span) {
  if (!r || !r->data || !aligned16(r->data)) return kStatusInvalid;
  for (long long s : {r->row_stride, r->head_stride})
    if (s < 0 || s >= (1ll << 38)) return kStatusInvalid;
  Dim dims[2] = {{rows, r->row_stride * 2}, {heads, r->head_stride * 2}};
  if (!strides_ok(dims, 2, static_cast<int64_t>(d) * 2, output)) return kStatusInvalid;
  *out = {static_cast<uint8_t*>(r->data), dims[0].stride, dims[1].stride};
  *span = {r->data, span_of(dims, 2, static_cast<int64_t>(d) * 2)};
  return kStatusOk;
}

int paged_device(PagedKv* kv, int** status) {
  int dev = 0;
  const int rc = current_device(&dev);
  if (rc) return rc;
  *status = status_ptr(dev);
  kv->check = check_ptr(dev);
  return *status && kv->check ? kStatusOk : kStatusCuda;
}

int paged_append_entry(const attn_paged_kv_t* c, const attn_rows_t* k, const attn_rows_t* v, const attn_rows_t* q,
                       const attn_rows_t* q_out, int q_heads, int rows, const int* token_start, const float* cos,
                       const float* sin, int table_rows, int rot_dim, int interleaved, int x_type, void* stream) {
  PagedAppendArgs a = {};
  Span ks, vs, kn, vn, qn = {}, qo = {};
  int rc = paged_kv(c, x_type, &a.kv, &ks, &vs);
  if (rc) return rc;
  if (rows < 0 || q_heads < 0 || rot_dim < 0) return kStatusInvalid;
  if (!token_start && rows != c->B) return kStatusInvalid;
  if ((q == nullptr) != (q_heads == 0) || (q == nullptr) != (q_out == nullptr)) return kStatusInvalid;
  if (rows > (1 << 30) || q_heads > 65535) return kStatusUnsupported;
  if (rot_dim % 16 || rot_dim > c->head_dim) return kStatusUnsupported;
  if (rot_dim && (!cos || !sin || table_rows < 1 || !aligned16(cos) || !aligned16(sin))) return kStatusInvalid;
  if (reinterpret_cast<uintptr_t>(token_start) & 3u) return kStatusInvalid;
  if (rows == 0) {
    t_last_launches = 0;
    return kStatusOk;
  }
  if ((rc = paged_rows(k, rows, c->kv_heads, c->head_dim, false, &a.k, &kn))) return rc;
  if ((rc = paged_rows(v, rows, c->kv_heads, c->head_dim, false, &a.v, &vn))) return rc;
  if (q) {
    if ((rc = paged_rows(q, rows, q_heads, c->head_dim, false, &a.q, &qn))) return rc;
    if ((rc = paged_rows(q_out, rows, q_heads, c->head_dim, true, &a.q_out, &qo))) return rc;
    // q may be rotated in place (k and v may then lie between its rows)
    const bool in_place = a.q.p == a.q_out.p && a.q.row == a.q_out.row && a.q.head == a.q_out.head;
    if (!in_place && any_overlap(qo, {qn, kn, vn})) return kStatusInvalid;
  }
  const Span ts = {token_start, (static_cast<size_t>(c->B) + 1) * 4};
  const size_t tb = static_cast<size_t>(rot_dim ? table_rows : 0) * (rot_dim / 2) * 4;
  const Span lens = {c->seq_lens, static_cast<size_t>(c->B) * 4}, cs = {tb ? cos : nullptr, tb}, sn = {tb ? sin : nullptr, tb};
  const Span table = {c->block_table, (static_cast<size_t>(c->B - 1) * c->table_stride + c->max_pages) * 4};
  const size_t sum = static_cast<size_t>(c->num_pages) * c->kv_heads * c->head_dim * type_bytes(c->type);
  for (const Span& out : {ks, vs, Span{c->k_min, sum}, Span{c->k_max, sum}})
    if (any_overlap(out, {kn, vn, qn, qo, ts, lens, cs, sn, table})) return kStatusInvalid;
  if (any_overlap(qo, {ts, lens, cs, sn, table})) return kStatusInvalid;
  a.Hq = q_heads;
  a.rows = rows;
  a.token_start = token_start;
  a.cos = cos;
  a.sin = sin;
  a.table_rows = table_rows;
  a.rot = rot_dim;
  a.interleaved = interleaved ? 1 : 0;
  a.x_type = x_type;
  a.stream = static_cast<cudaStream_t>(stream);
  int* status = nullptr;
  if ((rc = paged_device(&a.kv, &status))) return rc;
  int launches = 0;
  if ((rc = launch_paged_append(a, &launches)) == kStatusOk) t_last_launches = launches;
  return rc;
}

int paged_decode_entry(const attn_paged_kv_t* c, const attn_rows_t* q, int q_heads, void* o, float* lse,
                       const int* pages, int n_pages, float scale, int x_type, void* workspace, void* stream) {
  PagedDecodeArgs a = {};
  Span ks, vs, qn;
  int rc = paged_kv(c, x_type, &a.kv, &ks, &vs);
  if (rc) return rc;
  if (!o || !lse || !std::isfinite(scale) || !aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return kStatusInvalid;
  // Logits in units of log2; an infinite factor would make NaN of products that are 0.
  const float sl2 = scale * c->k_scale * 1.4426950408889634f;
  if (!std::isfinite(sl2)) return kStatusInvalid;
  if (pages && (n_pages < 1 || (reinterpret_cast<uintptr_t>(pages) & 3u))) return kStatusInvalid;
  if ((rc = query_heads_ok(q_heads, c->B, c->kv_heads))) return rc;
  if (pages && !listed_pages_ok(n_pages, c->page_size)) return kStatusUnsupported;
  if ((rc = paged_rows(q, c->B, q_heads, c->head_dim, false, &a.q, &qn))) return rc;
  const int64_t need = paged_decode_workspace(c->B, q_heads, c->kv_heads, c->head_dim, c->page_size,
                                              pages ? n_pages : c->max_pages);
  if (need && (!workspace || !aligned16(workspace))) return kStatusInvalid;
  const size_t obytes = static_cast<size_t>(c->B) * q_heads * c->head_dim * 2, lbytes = static_cast<size_t>(c->B) * q_heads * 4;
  const Span list = {pages, pages ? static_cast<size_t>(c->B) * c->kv_heads * n_pages * 4 : 0};
  const Span table = {c->block_table, (static_cast<size_t>(c->B - 1) * c->table_stride + c->max_pages) * 4};
  const Span lens = {c->seq_lens, static_cast<size_t>(c->B) * 4};
  const Span outs[3] = {{o, obytes}, {lse, lbytes}, {need ? workspace : nullptr, static_cast<size_t>(need)}};
  for (int i = 0; i < 3; ++i) {
    if (any_overlap(outs[i], {ks, vs, qn, list, table, lens})) return kStatusInvalid;
    if (any_overlap(outs[i], {outs[(i + 1) % 3]})) return kStatusInvalid;
  }
  a.Hq = q_heads;
  a.o = static_cast<uint8_t*>(o);
  a.lse = lse;
  a.pages = pages;
  a.n_pages = n_pages;
  a.sl2 = sl2;
  a.x_type = x_type;
  a.stream = static_cast<cudaStream_t>(stream);
  a.ws = static_cast<uint8_t*>(workspace);
  if ((rc = paged_device(&a.kv, &a.status))) return rc;
  int launches = 0;
  if ((rc = launch_paged_decode(a, &launches)) == kStatusOk) t_last_launches = launches;
  return rc;
}

int paged_select_entry(const attn_paged_kv_t* c, const attn_rows_t* q, int q_heads, int* pages, int n_select,
                       int keep_first, int keep_last, int x_type, void* workspace, void* stream) {
  PagedSelectArgs a = {};
  Span ks, vs, qn;
  int rc = paged_kv(c, x_type, &a.kv, &ks, &vs);
  if (rc) return rc;
  if (!c->k_min || !pages || (reinterpret_cast<uintptr_t>(pages) & 3u)) return kStatusInvalid;
  if (n_select < 1 || keep_first < 0 || keep_last < 0 || static_cast<int64_t>(keep_first) + keep_last > n_select)
    return kStatusInvalid;
  if ((rc = query_heads_ok(q_heads, c->B, c->kv_heads))) return rc;
  if (!listed_pages_ok(n_select, c->page_size)) return kStatusUnsupported;
  if ((rc = paged_rows(q, c->B, q_heads, c->head_dim, false, &a.q, &qn))) return rc;
  const int64_t need = paged_select_workspace(c->B, c->kv_heads, c->max_pages);
  if (need && (!workspace || !aligned16(workspace))) return kStatusInvalid;
  const size_t sum = static_cast<size_t>(c->num_pages) * c->kv_heads * c->head_dim * type_bytes(c->type);
  const Span table = {c->block_table, (static_cast<size_t>(c->B - 1) * c->table_stride + c->max_pages) * 4};
  const Span lens = {c->seq_lens, static_cast<size_t>(c->B) * 4};
  const Span out = {pages, static_cast<size_t>(c->B) * c->kv_heads * n_select * 4};
  const Span ws = {need ? workspace : nullptr, static_cast<size_t>(need)};
  for (const Span& s : {out, ws})
    if (any_overlap(s, {qn, Span{c->k_min, sum}, Span{c->k_max, sum}, ks, vs, table, lens})) return kStatusInvalid;
  if (any_overlap(out, {ws})) return kStatusInvalid;
  a.Hq = q_heads;
  a.pages = pages;
  a.n_select = n_select;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  a.x_type = x_type;
  a.stream = static_cast<cudaStream_t>(stream);
  a.ws = static_cast<uint8_t*>(workspace);
  int* status = nullptr;
  if ((rc = paged_device(&a.kv, &status))) return rc;
  int launches = 0;
  if ((rc = launch_paged_select(a, &launches)) == kStatusOk) t_last_launches = launches;
  return rc;
}

}  // namespace
}  // namespace attn

extern "C" {

int attn_paged_append(const attn_paged_kv_t* kv, const attn_rows_t* k, const attn_rows_t* v, const attn_rows_t* q,
                      const attn_rows_t* q_out, int q_heads, int rows, const int* token_start, const float* cos,
                      const float* sin, int table_rows, int rot_dim, int interleaved, int x_type, void* stream) {
  return attn::paged_append_entry(kv, k, v, q, q_out, q_heads, rows, token_start, cos, sin, table_rows, rot_dim,
                                  interleaved, x_type, stream);
}

int attn_paged_decode(const attn_paged_kv_t* kv, const attn_rows_t* q, int q_heads, void* o, float* lse,
                      const int* pages, int n_pages, float scale, int x_type, void* workspace, void* stream) {
  return attn::paged_decode_entry(kv, q, q_heads, o, lse, pages, n_pages, scale, x_type, workspace, stream);
}

int attn_paged_select(const attn_paged_kv_t* kv, const attn_rows_t* q, int q_heads, int* pages, int n_select,
                      int keep_first, int keep_last, int x_type, void* workspace, void* stream) {
  return attn::paged_select_entry(kv, q, q_heads, pages, n_select, keep_first, keep_last, x_type, workspace, stream);
}

long long attn_paged_decode_workspace(const attn_paged_kv_t* kv, int q_heads, int n_pages) {
  if (!kv || attn::paged_sizes(kv) || attn::query_heads_ok(q_heads, kv->B, kv->kv_heads) ||
      (n_pages >= 1 && !attn::listed_pages_ok(n_pages, kv->page_size)))
    return 0;
  return attn::paged_decode_workspace(kv->B, q_heads, kv->kv_heads, kv->head_dim, kv->page_size,
                                      n_pages < 1 ? kv->max_pages : n_pages);
}

long long attn_paged_select_workspace(const attn_paged_kv_t* kv) {
  if (!kv || attn::paged_sizes(kv)) return 0;
  return attn::paged_select_workspace(kv->B, kv->kv_heads, kv->max_pages);
}

}  // extern "C"

extern "C" {

int attn_fwd_dropout(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                     int H, int N, int d, float scale, int causal, float p_drop,
                     unsigned long long seed, unsigned int offset, void* stream) {
  attn::DropParams dr;
  const int rc = attn::make_drop(p_drop, seed, offset, &dr);
  if (rc) return rc;
  return attn::fwd_entry(q, k, v, o, lse, B, H, N, d, scale, causal, stream, true, dr);
}

int attn_fwd_dropout_f16(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                         int H, int N, int d, float scale, int causal, float p_drop,
                         unsigned long long seed, unsigned int offset, void* stream) {
  attn::DropParams dr;
  const int rc = attn::make_drop(p_drop, seed, offset, &dr);
  if (rc) return rc;
  return attn::fwd_entry(q, k, v, o, lse, B, H, N, d, scale, causal, stream, false, dr);
}

int attn_bwd_dropout(const void* q, const void* k, const void* v, const void* o, const void* dO,
                     const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                     float scale, int causal, float p_drop, unsigned long long seed,
                     unsigned int offset, void* stream) {
  attn::DropParams dr;
  const int rc = attn::make_drop(p_drop, seed, offset, &dr);
  if (rc) return rc;
  return attn::bwd_entry(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, stream, true, dr);
}

int attn_bwd_dropout_f16(const void* q, const void* k, const void* v, const void* o, const void* dO,
                         const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                         float scale, int causal, float p_drop, unsigned long long seed,
                         unsigned int offset, void* stream) {
  attn::DropParams dr;
  const int rc = attn::make_drop(p_drop, seed, offset, &dr);
  if (rc) return rc;
  return attn::bwd_entry(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, stream, false, dr);
}

int attn_fwd_fp8(const void* q, const void* k, const void* v, float descale_q, float descale_k,
                 float descale_v, void* o, float* lse, int B, int H, int N, int d, float scale,
                 int causal, void* stream) {
  return attn::fp8_entry(q, k, v, descale_q, descale_k, descale_v, o, lse, B, H, N, d, scale, causal,
                         stream);
}

}  // extern "C"

namespace attn {
namespace {
int blocksparse_bwd_entry(const void* q, const void* k, const void* v, const void* o, const void* dO,
                          const float* lse, void* dq, void* dk, void* dv, const unsigned char* block_mask,
                          int mask_heads, int B, int H, int N, int d, float scale, int causal, void* stream,
                          bool bf16, const DropParams& drop = kNoDrop) {
  if (!block_mask) return kStatusInvalid;
  if (mask_heads != 1 && mask_heads != H) return kStatusInvalid;
  if (N > 0 && (N + 127) / 128 > kMaxSparseTiles) return kStatusUnsupported;
  return bwd_entry(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, stream, bf16, drop,
                   block_mask, mask_heads);
}
}  // namespace
}  // namespace attn

extern "C" {

int attn_bwd_blocksparse(const void* q, const void* k, const void* v, const void* o, const void* dO,
                         const float* lse, void* dq, void* dk, void* dv,
                         const unsigned char* block_mask, int mask_heads, int B, int H, int N, int d,
                         float scale, int causal, void* stream) {
  return attn::blocksparse_bwd_entry(q, k, v, o, dO, lse, dq, dk, dv, block_mask, mask_heads, B, H, N, d,
                                     scale, causal, stream, true);
}

int attn_bwd_blocksparse_f16(const void* q, const void* k, const void* v, const void* o, const void* dO,
                             const float* lse, void* dq, void* dk, void* dv,
                             const unsigned char* block_mask, int mask_heads, int B, int H, int N, int d,
                             float scale, int causal, void* stream) {
  return attn::blocksparse_bwd_entry(q, k, v, o, dO, lse, dq, dk, dv, block_mask, mask_heads, B, H, N, d,
                                     scale, causal, stream, false);
}

int attn_fwd_blocksparse(const void* q, const void* k, const void* v, void* o, float* lse,
                         const unsigned char* block_mask, int mask_heads, int B, int H, int N, int d,
                         float scale, int causal, void* stream) {
  return attn::blocksparse_entry(q, k, v, o, lse, block_mask, mask_heads, B, H, N, d, scale, causal,
                                 stream, true);
}

int attn_fwd_blocksparse_f16(const void* q, const void* k, const void* v, void* o, float* lse,
                             const unsigned char* block_mask, int mask_heads, int B, int H, int N, int d,
                             float scale, int causal, void* stream) {
  return attn::blocksparse_entry(q, k, v, o, lse, block_mask, mask_heads, B, H, N, d, scale, causal,
                                 stream, false);
}

int attn_fwd_blocksparse_dropout(const void* q, const void* k, const void* v, void* o, float* lse,
                                 const unsigned char* block_mask, int mask_heads, int B, int H, int N, int d,
                                 float scale, int causal, float p_drop, unsigned long long seed,
                                 unsigned int offset, void* stream) {
  attn::DropParams dr;
  const int rc = attn::make_drop(p_drop, seed, offset, &dr);
  if (rc) return rc;
  return attn::blocksparse_entry(q, k, v, o, lse, block_mask, mask_heads, B, H, N, d, scale, causal,
                                 stream, true, dr);
}

int attn_fwd_blocksparse_dropout_f16(const void* q, const void* k, const void* v, void* o, float* lse,
                                     const unsigned char* block_mask, int mask_heads, int B, int H, int N,
                                     int d, float scale, int causal, float p_drop, unsigned long long seed,
                                     unsigned int offset, void* stream) {
  attn::DropParams dr;
  const int rc = attn::make_drop(p_drop, seed, offset, &dr);
  if (rc) return rc;
  return attn::blocksparse_entry(q, k, v, o, lse, block_mask, mask_heads, B, H, N, d, scale, causal,
                                 stream, false, dr);
}

int attn_bwd_blocksparse_dropout(const void* q, const void* k, const void* v, const void* o, const void* dO,
                                 const float* lse, void* dq, void* dk, void* dv,
                                 const unsigned char* block_mask, int mask_heads, int B, int H, int N, int d,
                                 float scale, int causal, float p_drop, unsigned long long seed,
                                 unsigned int offset, void* stream) {
  attn::DropParams dr;
  const int rc = attn::make_drop(p_drop, seed, offset, &dr);
  if (rc) return rc;
  return attn::blocksparse_bwd_entry(q, k, v, o, dO, lse, dq, dk, dv, block_mask, mask_heads, B, H, N, d,
                                     scale, causal, stream, true, dr);
}

int attn_bwd_blocksparse_dropout_f16(const void* q, const void* k, const void* v, const void* o,
                                     const void* dO, const float* lse, void* dq, void* dk, void* dv,
                                     const unsigned char* block_mask, int mask_heads, int B, int H, int N,
                                     int d, float scale, int causal, float p_drop, unsigned long long seed,
                                     unsigned int offset, void* stream) {
  attn::DropParams dr;
  const int rc = attn::make_drop(p_drop, seed, offset, &dr);
  if (rc) return rc;
  return attn::blocksparse_bwd_entry(q, k, v, o, dO, lse, dq, dk, dv, block_mask, mask_heads, B, H, N, d,
                                     scale, causal, stream, false, dr);
}

int attn_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                int L, int d, float scale, void* stream) {
  return attn::decode_entry(q, k, v, o, lse, B, H, L, d, scale, stream);
}

int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
             int N, int d, float scale, int causal, void* stream) {
  return attn::fwd_entry(q, k, v, o, lse, B, H, N, d, scale, causal, stream, true);
}

int attn_fwd_f16(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                 int N, int d, float scale, int causal, void* stream) {
  return attn::fwd_entry(q, k, v, o, lse, B, H, N, d, scale, causal, stream, false);
}

int attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO,
             const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
             float scale, int causal, void* stream) {
  return attn::bwd_entry(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, stream, true);
}

int attn_bwd_f16(const void* q, const void* k, const void* v, const void* o, const void* dO,
                 const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                 float scale, int causal, void* stream) {
  return attn::bwd_entry(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, stream, false);
}

int attn_sync_status(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return attn::kStatusCuda;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return attn::kStatusCuda;
  int value = 0, check = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbol(&value, g_attn_status, sizeof(int)) != cudaSuccess) return attn::kStatusCuda;
  if (value != 0 && cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(int)) != cudaSuccess)
    return attn::kStatusCuda;
  if (cudaMemcpyFromSymbol(&check, g_attn_check, sizeof(int)) != cudaSuccess) return attn::kStatusCuda;
  if (check != 0 && cudaMemcpyToSymbol(g_attn_check, &zero, sizeof(int)) != cudaSuccess)
    return attn::kStatusCuda;
  return value ? value : check;
}

const char* attn_status_string(int status) {
  switch (status) {
    case ATTN_OK: return "ok";
    case ATTN_ERR_INVALID_ARG: return "invalid argument";
    case ATTN_ERR_UNSUPPORTED: return "unsupported configuration";
    case ATTN_ERR_CUDA: return "CUDA runtime error";
    case ATTN_ERR_TIMEOUT: return "device pipeline wait timed out";
    case ATTN_ERR_ARCH: return "device is not sm_103 (GB300)";
    case ATTN_ERR_DEVICE_CHECK: return "device-side check failed";
    default: return "unknown status";
  }
}

int attn_last_launch_count(void) { return attn::t_last_launches; }

}  // extern "C"
