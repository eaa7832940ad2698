// C-ABI of the exact-attention library: host-side validation, device check,
// TMA descriptor encoding and launches.  See include/attn47.h for the
// contract of every entry point.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <type_traits>
#include <utility>

#include "attn47.h"
#include "decode_kv4_sm103.h"
#include "decode_kv8_sm103.h"
#include "decode_sm103.h"
#include "bwd_sm103.h"
#include "fusion_sm103.h"
#include "gemm_sm103.h"
#include "fwd_sm103.h"
#include "kv4.cuh"
#include "kv8.cuh"
#include "rope_sm103.h"
#include "ssd_sm103.h"
#include "ptx.cuh"

// Per-device error word written by the kernels (ATTN_DEV_* bits).
__device__ unsigned int g_attn47_status;

// Fixed scratch of attn_decode_paged_noalloc: the partial results of
// sequences whose keys are split across CTAs.  Every device that loads the
// library holds it until the process exits; every call of that entry point
// on a device reuses it.
constexpr size_t kNoAllocScratchBytes = size_t(8) << 20;   // 8 MiB
static __device__ __align__(256) unsigned char g_attn47_noalloc_scratch[kNoAllocScratchBytes];

namespace {

thread_local char g_last_error[512] = "";

attn_status_t fail(attn_status_t s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return s;
}

unsigned long long g_timeout_ns = 1000000000ull;

int g_decode_max_ctas = 0;  // 0 = one full wave
std::atomic<int> g_decode_early_plan{0};

// Tags of the decode's per-run arrival counters: a different nonzero value
// for every call of this process, starting from a clock-derived value so
// that workspace contents left by another process are unlikely to carry it.
unsigned int next_decode_epoch() {
  static std::atomic<unsigned int> epoch{static_cast<unsigned int>(
      std::chrono::steady_clock::now().time_since_epoch().count() * 2654435761ull)};
  unsigned int e;
  do {
    e = epoch.fetch_add(1u) + 1u;
  } while (e == 0u);
  return e;
}

constexpr int kMaxDevices = 64;
struct DeviceInfo {
  int index = -1;
  bool checked = false;
  bool usable = false;
  int sms = 0;
  unsigned int* status = nullptr;
  void* noalloc_scratch = nullptr;   // device address of the fixed scratch array
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_mu;

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;
using AddressRangeFn = CUresult (*)(CUdeviceptr*, size_t*, CUdeviceptr);
AddressRangeFn g_address_range = nullptr;
using PointerAttributesFn = CUresult (*)(unsigned int, CUpointer_attribute*, void**, CUdeviceptr);
PointerAttributesFn g_pointer_attributes = nullptr;

// Current device, checked once: compute capability 10.3, status word address.
attn_status_t current_device(DeviceInfo** out) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess)
    return fail(ATTN_ERR_DEVICE, "no usable CUDA device: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(ATTN_ERR_DEVICE, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.checked) {
    int major = 0, minor = 0, sms = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    d.sms = sms;
    d.index = dev;
    if (major != 10 || minor != 3) {
      d.checked = true;
      d.usable = false;
      return fail(ATTN_ERR_DEVICE, "device %d is compute capability %d.%d; this library is built "
                  "for sm_103a (10.3) only", dev, major, minor);
    }
    void* addr = nullptr;
    e = cudaGetSymbolAddress(&addr, g_attn47_status);
    if (e != cudaSuccess)
      return fail(ATTN_ERR_DEVICE, "status word unavailable: %s", cudaGetErrorString(e));
    d.status = static_cast<unsigned int*>(addr);
    if (g_encode == nullptr) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
      if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || fn == nullptr)
        return fail(ATTN_ERR_DEVICE, "driver entry point cuTensorMapEncodeTiled not found");
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
    if (g_address_range == nullptr) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      e = cudaGetDriverEntryPointByVersion("cuMemGetAddressRange", &fn, 12000, cudaEnableDefault, &q);
      if (e == cudaSuccess && q == cudaDriverEntryPointSuccess && fn != nullptr)
        g_address_range = reinterpret_cast<AddressRangeFn>(fn);
      else
        cudaGetLastError();   // optional: without it only the memory type is checked
    }
    if (g_pointer_attributes == nullptr) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      e = cudaGetDriverEntryPointByVersion("cuPointerGetAttributes", &fn, 12000, cudaEnableDefault, &q);
      if (e == cudaSuccess && q == cudaDriverEntryPointSuccess && fn != nullptr)
        g_pointer_attributes = reinterpret_cast<PointerAttributesFn>(fn);
      else
        cudaGetLastError();   // optional: without it every check takes the longer way
    }
    d.usable = true;
    d.checked = true;
  }
  if (!d.usable) return fail(ATTN_ERR_DEVICE, "device %d is not a compute capability 10.3 GPU", dev);
  *out = &d;
  return ATTN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
bool finite_positive(float x) { return std::isfinite(x) && x > 0.f; }

// A buffer a kernel will read or write: `bytes` from `p` (p may be NULL when
// the argument is optional).
struct Buf {
  const void* p;
  size_t bytes;
  const char* name;
};

// Every buffer must be memory the current device owns (cudaMalloc'd, from a
// stream-ordered pool, or managed), and [p, p + bytes) must lie inside the
// allocation that holds p.  A host address (pageable or pinned) handed to
// TMA or to a kernel would be accessed as if it were device memory, and an
// undersized buffer would be overrun; both are refused here, before any
// launch, with ATTN_ERR_INVALID_ARG.
//
// One driver query answers for an ordinary buffer; whatever it does not
// clear goes through the separate queries, which name what is wrong.  (A
// decode step's small calls are bound by the host, and these checks were over
// half of their time in the library.)
bool buf_clears(const DeviceInfo& d, const Buf& b) {
  if (g_pointer_attributes == nullptr) return false;
  unsigned int type = 0, managed = 0;
  int ordinal = -1;
  CUdeviceptr base = 0;
  size_t size = 0;
  CUpointer_attribute attrs[5] = {CU_POINTER_ATTRIBUTE_MEMORY_TYPE, CU_POINTER_ATTRIBUTE_IS_MANAGED,
                                  CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL, CU_POINTER_ATTRIBUTE_RANGE_START_ADDR,
                                  CU_POINTER_ATTRIBUTE_RANGE_SIZE};
  void* out[5] = {&type, &managed, &ordinal, &base, &size};
  const uintptr_t p = reinterpret_cast<uintptr_t>(b.p);
  if (g_pointer_attributes(5, attrs, out, static_cast<CUdeviceptr>(p)) != CUDA_SUCCESS) return false;
  return type == CU_MEMORYTYPE_DEVICE && managed == 0 && ordinal == d.index && size != 0 && p >= base &&
         p - base <= size && b.bytes <= size - (p - base);
}

attn_status_t check_bufs(const DeviceInfo& d, std::initializer_list<Buf> bufs) {
  for (const Buf& b : bufs) {
    if (b.p == nullptr || b.bytes == 0 || buf_clears(d, b)) continue;
    cudaPointerAttributes attr;
    const cudaError_t e = cudaPointerGetAttributes(&attr, b.p);
    if (e != cudaSuccess) {
      cudaGetLastError();   // not a launch error: clear it
      return fail(ATTN_ERR_INVALID_ARG, "%s (%p) is not device memory: %s", b.name, b.p,
                  cudaGetErrorString(e));
    }
    const bool ok = attr.type == cudaMemoryTypeManaged ||
                    (attr.type == cudaMemoryTypeDevice && attr.device == d.index);
    if (!ok)
      return fail(ATTN_ERR_INVALID_ARG, "%s (%p) is not memory of device %d (memory type %d, device %d)",
                  b.name, b.p, d.index, (int)attr.type, attr.device);
    if (g_address_range != nullptr) {
      CUdeviceptr base = 0;
      size_t size = 0;
      if (g_address_range(&base, &size, reinterpret_cast<CUdeviceptr>(b.p)) == CUDA_SUCCESS) {
        const uintptr_t end = static_cast<uintptr_t>(base) + size;
        if (reinterpret_cast<uintptr_t>(b.p) + b.bytes > end)
          return fail(ATTN_ERR_INVALID_ARG, "%s: %zu bytes from %p run past the end of its allocation "
                      "(%zu bytes at %p)", b.name, b.bytes, b.p, size, reinterpret_cast<void*>(base));
      }
    }
  }
  return ATTN_OK;
}

// cuTensorMapEncodeTiled, 128-byte swizzle, zero fill out of bounds.  It wants a
// context, which a thread that has made no runtime call of consequence yet lacks: the
// current device's is bound to it then.
CUresult encode_tiled(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                      const cuuint64_t* strides, const cuuint32_t* box, const cuuint32_t* estr) {
  auto encode = [&]() {
    return g_encode(map, type, rank, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  int dev = 0;
  if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = encode();
  return r;
}

// bf16 tensor map over `rank` dims (innermost first), 64-column boxes,
// 128-byte swizzle, zero fill out of bounds.
attn_status_t encode_bf16(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                          const cuuint32_t* box) {
  cuuint64_t strides[4];
  cuuint64_t acc = dims[0] * 2;
  for (int i = 1; i < rank; ++i) {
    strides[i - 1] = acc;
    acc *= dims[i];
  }
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, base, dims, strides, box, estr);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_INVALID_ARG, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return ATTN_OK;
}

// bf16 tensor map with explicit byte strides of dims 1.. (innermost dim
// contiguous), 128-byte swizzle, zero fill out of bounds.
attn_status_t encode_bf16_strided(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                                  const cuuint64_t* strides, const cuuint32_t* box) {
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, base, dims, strides, box, estr);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_INVALID_ARG, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return ATTN_OK;
}

attn_status_t launch_result(cudaError_t e, const char* what) {
  if (e != cudaSuccess) {
    cudaGetLastError();   // reported here: not left for another call to find
    return fail(ATTN_ERR_LAUNCH, "%s launch failed: %s", what, cudaGetErrorString(e));
  }
  g_last_error[0] = '\0';
  return ATTN_OK;
}

// Host-side checks of a decode call that need neither the workspace nor the
// device: sizes, supported shapes, null and misaligned pointers.  Shared by
// attn_decode_paged and attn_decode_paged_noalloc.
attn_status_t decode_check_args(const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* block_table, const int32_t* seq_lens, int num_seqs,
                                int Hq, int Hkv, int d, int block_size, int max_blocks_per_seq,
                                int num_blocks, float scale, const void* o, const float* lse) {
  if (num_seqs < 0 || Hq < 1 || Hkv < 1 || max_blocks_per_seq < 1 || num_blocks < 1)
    return fail(ATTN_ERR_INVALID_ARG,
                "sizes must satisfy num_seqs >= 0, Hq, Hkv, max_blocks_per_seq, num_blocks >= 1");
  if (Hq % Hkv != 0) return fail(ATTN_ERR_INVALID_ARG, "Hq (%d) is not a multiple of Hkv (%d)", Hq, Hkv);
  if (!finite_positive(scale)) return fail(ATTN_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (block_size != 16) return fail(ATTN_ERR_UNSUPPORTED, "block_size %d not supported (16)", block_size);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", d);
  if (Hq / Hkv > 16) return fail(ATTN_ERR_UNSUPPORTED, "Hq/Hkv = %d > 16 not supported", Hq / Hkv);
  if (static_cast<long long>(num_blocks) * Hkv * block_size >= 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "KV pool too large (num_blocks * Hkv * 16 >= 2^31)");
  if (static_cast<long long>(max_blocks_per_seq) * block_size >= 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "max_blocks_per_seq too large");
  if (static_cast<long long>(num_seqs) * Hq >= 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "num_seqs * Hq too large");
  if (num_seqs == 0) return ATTN_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !o)
    return fail(ATTN_ERR_INVALID_ARG, "q, caches, block_table, seq_lens and o must be non-null");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o))
    return fail(ATTN_ERR_INVALID_ARG, "q, caches and o must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(ATTN_ERR_INVALID_ARG, "block_table, seq_lens and lse must be 4-byte aligned");
  return ATTN_OK;
}

// Bytes of every decode buffer other than the workspace.
struct DecodeBytes {
  size_t q, cache, table, lens, o, lse;
};
DecodeBytes decode_bytes(int num_seqs, int Hq, int Hkv, int d, int max_blocks, int num_blocks) {
  DecodeBytes b;
  b.q = b.o = static_cast<size_t>(num_seqs) * Hq * d * 2;
  b.cache = static_cast<size_t>(num_blocks) * Hkv * 16 * d * 2;
  b.table = static_cast<size_t>(num_seqs) * max_blocks * 4;
  b.lens = static_cast<size_t>(num_seqs) * 4;
  b.lse = static_cast<size_t>(num_seqs) * Hq * 4;
  return b;
}

// Checks the decode's buffers against the device, encodes the cache maps and
// launches the decode with a workspace that has already been checked.
attn_status_t decode_launch(const DeviceInfo& dev, const void* q, const void* k_cache,
                            const void* v_cache, const int32_t* block_table, const int32_t* seq_lens,
                            int num_seqs, int Hq, int Hkv, int d, int max_blocks_per_seq, int num_blocks,
                            float scale, void* o, float* lse, void* workspace, void* stream) {
  const DecodeBytes nb = decode_bytes(num_seqs, Hq, Hkv, d, max_blocks_per_seq, num_blocks);
  attn_status_t st = check_bufs(dev, {{q, nb.q, "q"}, {k_cache, nb.cache, "k_cache"},
                                      {v_cache, nb.cache, "v_cache"}, {block_table, nb.table, "block_table"},
                                      {seq_lens, nb.lens, "seq_lens"}, {o, nb.o, "o"}, {lse, nb.lse, "lse"}});
  if (st != ATTN_OK) return st;
  // One copy per (block, head) slice: 64 columns x 16 rows x d/64 halves.
  const cuuint32_t box[3] = {64, 16, static_cast<cuuint32_t>(d / 64)};
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(num_blocks) * Hkv * 16,
                              static_cast<cuuint64_t>(d / 64)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, 128};
  alignas(64) CUtensorMap tk, tv;
  if ((st = encode_bf16_strided(&tk, k_cache, 3, dims, strides, box)) != ATTN_OK) return st;
  if ((st = encode_bf16_strided(&tv, v_cache, 3, dims, strides, box)) != ATTN_OK) return st;

  attn47::DecLaunch a;
  a.tk = &tk;
  a.tv = &tv;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.o = o;
  a.lse = lse;
  a.workspace = static_cast<float*>(workspace);
  a.num_seqs = num_seqs;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.sms = dev.sms;
  a.max_ctas = g_decode_max_ctas;
  a.early_plan = g_decode_early_plan.load();
  a.epoch = next_decode_epoch();
  a.scale = scale;
  a.status = dev.status;
  a.timeout_ns = g_timeout_ns;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_result(attn47::launch_decode_sm103(a), "attn_decode_paged");
}

// Most token rows of one launch of the kernels that take a warp per row (they
// count in 32 bits).
constexpr long long kMaxTokens = 0x7f000000LL;

// ------------------------------------------------------ rows given by strides
// Elements from the first to one past the last of a view.
long long heads_extent(const attn_heads_t& h, int B, int N, int d) {
  return (B - 1) * h.stride_batch + (N - 1) * h.stride_token + (h.heads - 1) * h.stride_head + d;
}

attn_status_t check_heads(const attn_heads_t* h, const char* name, int B, int N, int d, bool output) {
  if (h == nullptr || h->data == nullptr) return fail(ATTN_ERR_INVALID_ARG, "%s must be non-null", name);
  if (h->heads < 1) return fail(ATTN_ERR_INVALID_ARG, "%s must have heads >= 1", name);
  if (!aligned16(h->data)) return fail(ATTN_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  struct {
    long long stride, n;
  } dim[3] = {{h->stride_batch, B}, {h->stride_token, N}, {h->stride_head, h->heads}};
  for (const auto& x : dim) {
    if (x.stride < 0 || x.stride % 8 != 0)
      return fail(ATTN_ERR_INVALID_ARG, "%s: strides must be non-negative multiples of 8 elements", name);
    if (x.n > 1 && x.stride > (1LL << 46) / x.n) return fail(ATTN_ERR_INVALID_ARG, "%s: stride too large", name);
    if (&x != dim && x.n > 1 && x.stride >= (1LL << 34))
      return fail(ATTN_ERR_UNSUPPORTED, "%s: token or head stride of 2^34 elements or more not supported", name);
  }
  if (output) {
    // No two rows may share an element: taken from the smallest stride up,
    // each stride spans all that lies inside it.
    for (int i = 0; i < 3; ++i)
      for (int j = i + 1; j < 3; ++j)
        if (dim[j].stride < dim[i].stride) std::swap(dim[i], dim[j]);
    long long inner = d;
    for (const auto& x : dim) {
      if (x.n == 1) continue;
      if (x.stride < inner) return fail(ATTN_ERR_INVALID_ARG, "%s: rows overlap each other", name);
      inner += (x.n - 1) * x.stride;
    }
  }
  return ATTN_OK;
}

bool heads_identical(const attn_heads_t& a, const attn_heads_t& b, int B, int N) {
  return a.data == b.data && a.heads == b.heads && (B == 1 || a.stride_batch == b.stride_batch) &&
         (N == 1 || a.stride_token == b.stride_token) && (a.heads == 1 || a.stride_head == b.stride_head);
}

// Memory by strides, in bytes: runs of `run` bytes, n[i] of them stride[i] apart
// in each of three dimensions.
struct Strided {
  const void* p;
  long long run;
  long long stride[3], n[3];
};

Strided strided(const attn_heads_t& h, int B, int N, int d) {
  return Strided{h.data, 2LL * d, {2 * h.stride_batch, 2 * h.stride_token, 2 * h.stride_head}, {B, N, h.heads}};
}

Strided flat(const void* p, size_t bytes) {
  return Strided{p, static_cast<long long>(bytes), {0, 0, 0}, {1, 1, 1}};
}

// Whether `off` = sum over the dimensions of m step with m in lo .. hi, give or
// take what two runs reach (lo_run .. hi_run).  Dimensions go from the largest
// step down, so that few m are left to try where they lie inside one another;
// `tries` bounds them elsewhere (then: yes).
struct Meeting {
  struct Dim {
    long long step, lo, hi;
  } dim[6];
  int dims = 0, tries = 4096;
  long long lo_run, hi_run;

  void add(long long step, long long lo, long long hi) {
    if (step == 0 || lo == hi) return;
    int i = 0;
    while (i < dims && dim[i].step > step) ++i;
    if (i < dims && dim[i].step == step) {
      dim[i].lo += lo;
      dim[i].hi += hi;
      return;
    }
    for (int j = dims++; j > i; --j) dim[j] = dim[j - 1];
    dim[i] = Dim{step, lo, hi};
  }
  bool search(long long off, int i) {
    if (--tries < 0) return true;
    if (i == dims) return off >= lo_run && off <= hi_run;
    long long least = lo_run, most = hi_run;     // of all that comes after dimension i
    for (int j = i + 1; j < dims; ++j) {
      least += dim[j].lo * dim[j].step;
      most += dim[j].hi * dim[j].step;
    }
    const Dim& x = dim[i];
    auto floor_div = [&](long long v) { return v >= 0 ? v / x.step : -((-v + x.step - 1) / x.step); };
    long long m = -floor_div(most - off), last = floor_div(off - least);   // least <= off - m step <= most
    if (m < x.lo) m = x.lo;
    if (last > x.hi) last = x.hi;
    for (; m <= last; ++m)
      if (search(off - m * x.step, i + 1)) return true;
    return false;
  }
};

// Whether two pieces of strided memory share a byte.
bool meet(const Strided& a, const Strided& b) {
  long long ea = a.run, eb = b.run;
  for (int i = 0; i < 3; ++i) {
    ea += (a.n[i] - 1) * a.stride[i];
    eb += (b.n[i] - 1) * b.stride[i];
  }
  if (!overlap(a.p, static_cast<size_t>(ea), b.p, static_cast<size_t>(eb))) return false;
  Meeting m;
  m.lo_run = -(b.run - 1);
  m.hi_run = a.run - 1;
  for (int i = 0; i < 3; ++i) {
    m.add(a.stride[i], 0, a.n[i] - 1);
    m.add(b.stride[i], -(b.n[i] - 1), 0);
  }
  return m.search(static_cast<long long>(reinterpret_cast<uintptr_t>(b.p)) -
                      static_cast<long long>(reinterpret_cast<uintptr_t>(a.p)), 0);
}

attn_status_t check_apart(const attn_heads_t* out, const char* out_name, const attn_heads_t* in,
                          const char* in_name, bool may_be_same, int B, int N, int d) {
  if (out == nullptr || in == nullptr) return ATTN_OK;
  if (may_be_same && heads_identical(*out, *in, B, N)) return ATTN_OK;
  if (meet(strided(*out, B, N, d), strided(*in, B, N, d)))
    return fail(ATTN_ERR_INVALID_ARG, "%s overlaps %s", out_name, in_name);
  return ATTN_OK;
}

attn47::HeadRows head_rows(const attn_heads_t* h) {
  attn47::HeadRows r;
  if (h != nullptr) {
    r.data = h->data;
    r.batch = h->stride_batch;
    r.token = h->stride_token;
    r.head = h->stride_head;
    r.heads = h->heads;
  }
  return r;
}

// Host-side checks of a rotation and its form for the kernels.
attn_status_t check_rope(const attn_rope_t* r, int B, int d, bool needs_positions, attn47::RopeSpec* out) {
  *out = attn47::RopeSpec();
  if (r == nullptr) return ATTN_OK;              // no rotation
  if (r->rot < 16 || r->rot > d || r->rot % 16 != 0)
    return fail(ATTN_ERR_UNSUPPORTED, "rot %d not supported (a multiple of 16, 16 .. %d)", r->rot, d);
  if (r->axes < 1 || r->axes > 4) return fail(ATTN_ERR_UNSUPPORTED, "axes %d not supported (1 .. 4)", r->axes);
  if (!r->inv_freq || (reinterpret_cast<uintptr_t>(r->inv_freq) & 3u))
    return fail(ATTN_ERR_INVALID_ARG, "inv_freq must be non-null and 4-byte aligned");
  if (r->positions == nullptr && (needs_positions || r->axes != 1))
    return fail(ATTN_ERR_INVALID_ARG, "the rotation's positions must be non-null");
  if (reinterpret_cast<uintptr_t>(r->positions) & 3u)
    return fail(ATTN_ERR_INVALID_ARG, "the rotation's positions must be 4-byte aligned");
  if (r->stride_axis < 0 || r->stride_batch < 0 || r->stride_axis > (1LL << 40) ||
      (B > 1 && r->stride_batch > (1LL << 46) / B))
    return fail(ATTN_ERR_INVALID_ARG, "position strides must be non-negative and not too large");
  out->inv_freq = r->inv_freq;
  out->rot = r->rot;
  out->interleaved = r->interleaved != 0;
  out->positions = r->positions;
  out->axis_stride = r->stride_axis;
  out->batch_stride = r->stride_batch;
  if (r->pair_axis != nullptr) {
    for (int i = 0; i < r->rot / 2; ++i) {
      if (r->pair_axis[i] >= r->axes)
        return fail(ATTN_ERR_INVALID_ARG, "pair_axis[%d] = %d is not below axes (%d)", i, r->pair_axis[i], r->axes);
      out->pair_axis[i / 16] |= static_cast<uint32_t>(r->pair_axis[i]) << (2 * (i % 16));
    }
  }
  return ATTN_OK;
}

size_t rope_position_bytes(const attn_rope_t* r, int B, int N) {
  return static_cast<size_t>((r->axes - 1) * r->stride_axis + (B - 1) * r->stride_batch + N) * 4;
}

// What a call reads beside its rows.
struct Input {
  Strided s;
  const char* name;
};

// An output keeps off all of it: other warps may still be reading there.
attn_status_t check_inputs_kept(const Strided& out, const char* out_name, const Input* in, int n) {
  for (int i = 0; i < n; ++i)
    if (in[i].s.p != nullptr && meet(out, in[i].s))
      return fail(ATTN_ERR_INVALID_ARG, "%s overlaps %s", out_name, in[i].name);
  return ATTN_OK;
}

// The frequencies and positions of a rotation.
void rope_inputs(const attn_rope_t* r, int B, int N, Input (&in)[2]) {
  in[0] = Input{flat(r ? r->inv_freq : nullptr, r ? static_cast<size_t>(r->rot / 2) * 4 : 0), "inv_freq"};
  in[1] = Input{Strided{r ? r->positions : nullptr, 4LL * N, {r ? 4 * r->stride_axis : 0, r ? 4 * r->stride_batch : 0, 0},
                        {r ? r->axes : 1, B, 1}}, "the rotation's positions"};
}

attn_status_t rope_apply(const char* what, const attn_heads_t* q, const attn_heads_t* k, const attn_heads_t* q_out,
                         const attn_heads_t* k_out, const attn_rope_t* rope, int B, int N, int d, bool inverse,
                         void* stream) {
  if (B < 0 || N < 0) return fail(ATTN_ERR_INVALID_ARG, "sizes must satisfy B >= 0, N >= 0");
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", d);
  if (rope == nullptr) return fail(ATTN_ERR_INVALID_ARG, "rope must be non-null");
  const bool empty = B == 0 || N == 0;
  attn47::RopeLaunch a;
  attn_status_t st = check_rope(rope, B, d, !empty, &a.spec);
  if (st != ATTN_OK) return st;
  if (empty) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if ((st = check_heads(q, "q", B, N, d, false)) != ATTN_OK) return st;
  if ((st = check_heads(q_out, "q_out", B, N, d, true)) != ATTN_OK) return st;
  if (q->heads != q_out->heads) return fail(ATTN_ERR_INVALID_ARG, "q and q_out have different heads");
  if ((k == nullptr) != (k_out == nullptr))
    return fail(ATTN_ERR_INVALID_ARG, "k and k_out must both be given or both be NULL");
  if (k != nullptr) {
    if ((st = check_heads(k, "k", B, N, d, false)) != ATTN_OK) return st;
    if ((st = check_heads(k_out, "k_out", B, N, d, true)) != ATTN_OK) return st;
    if (k->heads != k_out->heads) return fail(ATTN_ERR_INVALID_ARG, "k and k_out have different heads");
  }
  if (static_cast<long long>(B) * N >= kMaxTokens)
    return fail(ATTN_ERR_UNSUPPORTED, "problem too large for one launch");
  if ((st = check_apart(q_out, "q_out", q, "q", true, B, N, d)) != ATTN_OK) return st;
  if ((st = check_apart(q_out, "q_out", k, "k", false, B, N, d)) != ATTN_OK) return st;
  if ((st = check_apart(k_out, "k_out", k, "k", true, B, N, d)) != ATTN_OK) return st;
  if ((st = check_apart(k_out, "k_out", q, "q", false, B, N, d)) != ATTN_OK) return st;
  if ((st = check_apart(k_out, "k_out", q_out, "q_out", false, B, N, d)) != ATTN_OK) return st;
  Input in[2];
  rope_inputs(rope, B, N, in);
  if ((st = check_inputs_kept(strided(*q_out, B, N, d), "q_out", in, 2)) != ATTN_OK) return st;
  if (k_out != nullptr && (st = check_inputs_kept(strided(*k_out, B, N, d), "k_out", in, 2)) != ATTN_OK) return st;
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != ATTN_OK) return st;
  auto bytes = [&](const attn_heads_t* h) { return h ? static_cast<size_t>(heads_extent(*h, B, N, d)) * 2 : 0; };
  if ((st = check_bufs(*dev, {{q->data, bytes(q), "q"}, {q_out->data, bytes(q_out), "q_out"},
                              {k ? k->data : nullptr, bytes(k), "k"},
                              {k_out ? k_out->data : nullptr, bytes(k_out), "k_out"},
                              {rope->inv_freq, static_cast<size_t>(rope->rot / 2) * 4, "inv_freq"},
                              {rope->positions, rope_position_bytes(rope, B, N), "positions"}})) != ATTN_OK)
    return st;
  a.spec.inverse = inverse;
  a.q = head_rows(q);
  a.k = head_rows(k);
  a.q_out = head_rows(q_out);
  a.k_out = head_rows(k_out);
  a.B = B;
  a.N = N;
  a.d = d;
  a.sms = dev->sms;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_result(attn47::launch_rope_sm103(a), what);
}

// All appends: into a cache of `bits` bits, 16 (k_cache and v_cache), 8 or 4
// (kv_cache, and with 4 the group).
attn_status_t rope_append(const char* what, int bits, const attn_heads_t* q, const attn_heads_t* k, const attn_heads_t* v,
                          const attn_heads_t* q_out, const attn_rope_t* rope, void* k_cache, void* v_cache,
                          void* kv_cache, int group, const int32_t* block_table, const int32_t* seq_ids,
                          const int32_t* positions, int T, int num_seqs, int d, int block_size,
                          int max_blocks_per_seq, int num_blocks, void* stream) {
  const bool packed = bits != 16;
  if (T < 0 || num_seqs < 1 || max_blocks_per_seq < 1 || num_blocks < 1)
    return fail(ATTN_ERR_INVALID_ARG, "sizes must satisfy T >= 0, num_seqs, max_blocks_per_seq, num_blocks >= 1");
  if (block_size != 16) return fail(ATTN_ERR_UNSUPPORTED, "block_size %d not supported (16)", block_size);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", d);
  if (static_cast<long long>(max_blocks_per_seq) * block_size >= 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "max_blocks_per_seq too large");
  if (T >= kMaxTokens) return fail(ATTN_ERR_UNSUPPORTED, "T too large");
  attn47::RopeAppendLaunch a;
  attn_status_t st = check_rope(rope, 1, d, false, &a.spec);
  if (st != ATTN_OK) return st;
  if (T == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if ((st = check_heads(k, "k", 1, T, d, false)) != ATTN_OK) return st;
  if ((st = check_heads(v, "v", 1, T, d, false)) != ATTN_OK) return st;
  if (k->heads != v->heads) return fail(ATTN_ERR_INVALID_ARG, "k and v have different heads");
  if ((q == nullptr) != (q_out == nullptr))
    return fail(ATTN_ERR_INVALID_ARG, "q and q_out must both be given or both be NULL");
  if (q != nullptr) {
    if ((st = check_heads(q, "q", 1, T, d, false)) != ATTN_OK) return st;
    if ((st = check_heads(q_out, "q_out", 1, T, d, true)) != ATTN_OK) return st;
    if (q->heads != q_out->heads) return fail(ATTN_ERR_INVALID_ARG, "q and q_out have different heads");
  }
  if (!block_table || !seq_ids || !positions)
    return fail(ATTN_ERR_INVALID_ARG, "block_table, seq_ids and positions must be non-null");
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_ids) & 3u) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u))
    return fail(ATTN_ERR_INVALID_ARG, "block_table, seq_ids and positions must be 4-byte aligned");
  const int Hkv = k->heads;
  if (packed ? (!kv_cache || !aligned16(kv_cache)) : (!k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache)))
    return fail(ATTN_ERR_INVALID_ARG, "the cache must be non-null and 16-byte aligned");
  const size_t cache = static_cast<size_t>(num_blocks) * Hkv *
                       (bits == 4   ? attn47::kv4_record_bytes_of(d, group)
                        : bits == 8 ? attn47::kv8_record_bytes_of(d)
                                    : static_cast<size_t>(16) * d * 2);
  if ((st = check_apart(q_out, "q_out", q, "q", true, 1, T, d)) != ATTN_OK) return st;
  if ((st = check_apart(q_out, "q_out", k, "k", false, 1, T, d)) != ATTN_OK) return st;
  if ((st = check_apart(q_out, "q_out", v, "v", false, 1, T, d)) != ATTN_OK) return st;
  if (!packed && overlap(k_cache, cache, v_cache, cache))
    return fail(ATTN_ERR_INVALID_ARG, "k_cache overlaps v_cache");
  const struct {
    const attn_heads_t* h;
    const char* name;
  } rows[] = {{q, "q"}, {k, "k"}, {v, "v"}, {q_out, "q_out"}};
  for (const auto& x : rows) {
    if (x.h == nullptr) continue;
    const size_t n = static_cast<size_t>(heads_extent(*x.h, 1, T, d)) * 2;
    if (packed ? overlap(kv_cache, cache, x.h->data, n)
            : overlap(k_cache, cache, x.h->data, n) || overlap(v_cache, cache, x.h->data, n))
      return fail(ATTN_ERR_INVALID_ARG, "%s overlaps the cache", x.name);
  }
  const size_t ints = static_cast<size_t>(T) * 4, table = static_cast<size_t>(num_seqs) * max_blocks_per_seq * 4;
  Input turn[2];
  rope_inputs(rope, 1, T, turn);
  const Input in[5] = {turn[0], turn[1], {flat(block_table, table), "block_table"}, {flat(seq_ids, ints), "seq_ids"},
                       {flat(positions, ints), "positions"}};
  if (q_out != nullptr && (st = check_inputs_kept(strided(*q_out, 1, T, d), "q_out", in, 5)) != ATTN_OK) return st;
  for (const void* x : {packed ? kv_cache : k_cache, packed ? nullptr : v_cache})
    if (x != nullptr && (st = check_inputs_kept(flat(x, cache), "the cache", in, 5)) != ATTN_OK) return st;
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != ATTN_OK) return st;
  auto bytes = [&](const attn_heads_t* h) { return h ? static_cast<size_t>(heads_extent(*h, 1, T, d)) * 2 : 0; };
  if ((st = check_bufs(*dev, {{q ? q->data : nullptr, bytes(q), "q"}, {k->data, bytes(k), "k"},
                              {v->data, bytes(v), "v"}, {q_out ? q_out->data : nullptr, bytes(q_out), "q_out"},
                              {k_cache, packed ? 0 : cache, "k_cache"}, {v_cache, packed ? 0 : cache, "v_cache"},
                              {kv_cache, packed ? cache : 0, "kv_cache"},
                              {block_table, table, "block_table"},
                              {seq_ids, ints, "seq_ids"}, {positions, ints, "positions"},
                              {rope ? rope->inv_freq : nullptr, rope ? static_cast<size_t>(rope->rot / 2) * 4 : 0,
                               "inv_freq"},
                              {rope ? rope->positions : nullptr, rope ? rope_position_bytes(rope, 1, T) : 0,
                               "the rotation's positions"}})) != ATTN_OK)
    return st;
  a.q = head_rows(q);
  a.k = head_rows(k);
  a.v = head_rows(v);
  a.q_out = head_rows(q_out);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.kv_cache = kv_cache;
  a.group = group;
  a.block_table = block_table;
  a.seq_ids = seq_ids;
  a.positions = positions;
  a.T = T;
  a.num_seqs = num_seqs;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.d = d;
  a.sms = dev->sms;
  a.status = dev->status;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_result(attn47::launch_rope_append_sm103(a), what);
}

// Read-back of a cache of `bits` bits, 8 or 4 (and then the group).
attn_status_t read_paged(const char* what, int bits, const void* kv_cache, int group, const int32_t* block_table,
                         const int32_t* seq_ids, const int32_t* positions, void* k, void* v, int T, int num_seqs,
                         int Hkv, int d, int block_size, int max_blocks_per_seq, int num_blocks, void* stream) {
  if (T < 0 || num_seqs < 1 || Hkv < 1 || max_blocks_per_seq < 1 || num_blocks < 1)
    return fail(ATTN_ERR_INVALID_ARG, "sizes must satisfy T >= 0, num_seqs, Hkv, max_blocks_per_seq, num_blocks >= 1");
  if (block_size != 16) return fail(ATTN_ERR_UNSUPPORTED, "block_size %d not supported (16)", block_size);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", d);
  if (static_cast<long long>(max_blocks_per_seq) * block_size >= 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "max_blocks_per_seq too large");
  if (T >= kMaxTokens) return fail(ATTN_ERR_UNSUPPORTED, "T too large");
  if (T == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if (!kv_cache || !block_table || !seq_ids || !positions || !k || !v)
    return fail(ATTN_ERR_INVALID_ARG, "kv_cache, block_table, seq_ids, positions, k and v must be non-null");
  if (!aligned16(kv_cache) || !aligned16(k) || !aligned16(v))
    return fail(ATTN_ERR_INVALID_ARG, "kv_cache, k and v must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_ids) & 3u) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u))
    return fail(ATTN_ERR_INVALID_ARG, "block_table, seq_ids and positions must be 4-byte aligned");
  const size_t cache = static_cast<size_t>(num_blocks) * Hkv *
                       (bits == 8 ? attn47::kv8_record_bytes_of(d) : attn47::kv4_record_bytes_of(d, group));
  const size_t out = static_cast<size_t>(T) * Hkv * d * 2;
  if (overlap(k, out, v, out) || overlap(k, out, kv_cache, cache) || overlap(v, out, kv_cache, cache))
    return fail(ATTN_ERR_INVALID_ARG, "k, v and kv_cache must not overlap");
  const size_t ints = static_cast<size_t>(T) * 4, table = static_cast<size_t>(num_seqs) * max_blocks_per_seq * 4;
  for (const void* x : {k, v})
    if (overlap(x, out, block_table, table) || overlap(x, out, seq_ids, ints) || overlap(x, out, positions, ints))
      return fail(ATTN_ERR_INVALID_ARG, "k and v must not overlap block_table, seq_ids or positions");
  DeviceInfo* dev = nullptr;
  attn_status_t st = current_device(&dev);
  if (st != ATTN_OK) return st;
  if ((st = check_bufs(*dev, {{kv_cache, cache, "kv_cache"}, {block_table, table, "block_table"},
                              {seq_ids, ints, "seq_ids"}, {positions, ints, "positions"}, {k, out, "k"},
                              {v, out, "v"}})) != ATTN_OK)
    return st;
  auto launch = [&](auto a) {
    a.kv_cache = kv_cache;
    a.block_table = block_table;
    a.seq_ids = seq_ids;
    a.positions = positions;
    a.k = k;
    a.v = v;
    a.T = T;
    a.Hkv = Hkv;
    a.d = d;
    a.num_seqs = num_seqs;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = num_blocks;
    a.sms = dev->sms;
    a.status = dev->status;
    a.stream = static_cast<cudaStream_t>(stream);
    if constexpr (std::is_same_v<decltype(a), attn47::Kv4ReadLaunch>) {
      a.group = group;
      return launch_result(attn47::launch_kv4_read_sm103(a), what);
    } else {
      return launch_result(attn47::launch_kv8_read_sm103(a), what);
    }
  };
  return bits == 8 ? launch(attn47::Kv8ReadLaunch()) : launch(attn47::Kv4ReadLaunch());
}

attn_status_t check_group(int group) {
  if (group != 32 && group != 64) return fail(ATTN_ERR_UNSUPPORTED, "group %d not supported (32 or 64)", group);
  return ATTN_OK;
}

// Host-side checks of attention over a cache of `bits` bits, 8 or 4 (and then the
// group), by N queries of each sequence: `need` bytes of workspace, `passes` over
// the blocks of a KV head.  *dev stays null where there is nothing to do.
attn_status_t check_quantised_attention(int bits, int group, bool decode, const void* q, const void* kv_cache,
                                        const int32_t* block_table, const int32_t* seq_lens, int num_seqs, int Hq,
                                        int Hkv, int N, int d, int block_size, int max_blocks_per_seq, int num_blocks,
                                        float scale, const void* o, const float* lse, const void* workspace,
                                        size_t workspace_bytes, size_t need, int passes, DeviceInfo** dev) {
  *dev = nullptr;
  if (num_seqs < 0 || Hq < 1 || Hkv < 1 || N < 0 || max_blocks_per_seq < 1 || num_blocks < 1)
    return fail(ATTN_ERR_INVALID_ARG,
                "sizes must satisfy num_seqs, N >= 0, Hq, Hkv, max_blocks_per_seq, num_blocks >= 1");
  if (Hq % Hkv != 0) return fail(ATTN_ERR_INVALID_ARG, "Hq (%d) is not a multiple of Hkv (%d)", Hq, Hkv);
  if (!finite_positive(scale)) return fail(ATTN_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (block_size != 16) return fail(ATTN_ERR_UNSUPPORTED, "block_size %d not supported (16)", block_size);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", d);
  if (decode && Hq / Hkv > 16) return fail(ATTN_ERR_UNSUPPORTED, "Hq/Hkv = %d > 16 not supported", Hq / Hkv);
  if (static_cast<long long>(max_blocks_per_seq) * block_size >= 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "max_blocks_per_seq too large");
  // The split counts blocks (and a few more units per run) in 32 bits.
  if (static_cast<__int128>(num_seqs) * Hq * N >= 0x7fffffff ||
      static_cast<__int128>(num_seqs) * Hkv * passes * (static_cast<long long>(max_blocks_per_seq) + 64) >= 0x7fffffff)
    return fail(ATTN_ERR_UNSUPPORTED, "problem too large for one launch");
  if (num_seqs == 0 || N == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if (!q || !kv_cache || !block_table || !seq_lens || !o || (need != 0 && !workspace))
    return fail(ATTN_ERR_INVALID_ARG, "q, kv_cache, block_table, seq_lens, o and workspace must be non-null");
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(o) || !aligned16(workspace))
    return fail(ATTN_ERR_INVALID_ARG, "q, kv_cache, o and workspace must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(ATTN_ERR_INVALID_ARG, "block_table, seq_lens and lse must be 4-byte aligned");
  if (workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  const size_t qb = static_cast<size_t>(num_seqs) * Hq * N * d * 2;
  const size_t cache = static_cast<size_t>(num_blocks) * Hkv *
                       (bits == 8 ? attn47::kv8_record_bytes_of(d) : attn47::kv4_record_bytes_of(d, group));
  const size_t table = static_cast<size_t>(num_seqs) * max_blocks_per_seq * 4, lens = static_cast<size_t>(num_seqs) * 4;
  const size_t lb = static_cast<size_t>(num_seqs) * Hq * N * 4;
  const struct {
    const void* p;
    size_t n;
  } others[] = {{q, qb}, {kv_cache, cache}, {block_table, table}, {seq_lens, lens}, {o, qb}, {lse, lse ? lb : 0}};
  for (const auto& x : others)
    if (need && x.n && overlap(workspace, need, x.p, x.n))
      return fail(ATTN_ERR_INVALID_ARG, "workspace overlaps an input or output of the attention");
  for (int i = 0; i < 4; ++i) {                  // (other warps may still be reading there)
    if (overlap(o, qb, others[i].p, others[i].n)) return fail(ATTN_ERR_INVALID_ARG, "o overlaps an input of the attention");
    if (lse && overlap(lse, lb, others[i].p, others[i].n))
      return fail(ATTN_ERR_INVALID_ARG, "lse overlaps an input of the attention");
  }
  if (lse && overlap(o, qb, lse, lb)) return fail(ATTN_ERR_INVALID_ARG, "o overlaps lse");
  attn_status_t st = current_device(dev);
  if (st == ATTN_OK)
    st = check_bufs(**dev, {{workspace, need, "workspace"}, {q, qb, "q"}, {kv_cache, cache, "kv_cache"},
                            {block_table, table, "block_table"}, {seq_lens, lens, "seq_lens"}, {o, qb, "o"},
                            {lse, lb, "lse"}});
  return st;
}

// What the launches of both decodes take alike.
template <class Launch>
void fill_quantised_decode(Launch& a, const DeviceInfo& dev, const void* q, const void* kv_cache,
                           const int32_t* block_table, const int32_t* seq_lens, int num_seqs, int Hq, int Hkv, int d,
                           int max_blocks_per_seq, int num_blocks, float scale, void* o, float* lse, void* workspace,
                           void* stream) {
  a.q = q;
  a.kv_cache = kv_cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.o = o;
  a.lse = lse;
  a.workspace = workspace;
  a.num_seqs = num_seqs;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  a.sms = dev.sms;
  a.device = dev.index;
  a.max_ctas = g_decode_max_ctas;
  a.epoch = next_decode_epoch();
  a.early_plan = g_decode_early_plan.load() > 0 ? 1 : 0;
  a.scale = scale;
  a.status = dev.status;
  a.timeout_ns = g_timeout_ns;
  a.stream = static_cast<cudaStream_t>(stream);
}

// Tensor map over the codes of 8-bit records, as 128-byte lines, a record's to a box,
// 128-byte swizzle.
attn_status_t encode_kv8(CUtensorMap* map, const void* base, cuuint64_t records, int d) {
  const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(d / 4), records};
  const cuuint64_t strides[2] = {128, attn47::kv8_record_bytes_of(d)};
  const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(d / 4), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, estr);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_INVALID_ARG, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return ATTN_OK;
}

// Whether an 8-bit prefill goes through the tiles of the forward kernel or, a group of
// query rows of a KV head at a time, through passes of the decode kernel.  Both take
// time in proportion to the lengths: for 1000 keys a wave of 152 CTAs about 20 us (d =
// 64: 17), a pass of one KV head of one sequence, split over all SMs, 42 ns (d = 64:
// 23, with three column tiles 31).  So as many passes as CTAs of all waves, times
// `share`, take as long as the tiles, which are taken beyond that.  Measured, passes
// against tiles: d = 128, 12 heads over 2 KV heads, 6000 keys, 4 sequences of 8 new
// tokens 29 and 121 us, of 128 121 and 121; 16 sequences of 32 121 and 125, of 64 217
// and 123; 32 heads over 8, 64 sequences of 8 new tokens and 1000 keys (4 waves) 68
// and 111, of 32 201 and 115; d = 64, 16 heads over 4, 6000 keys, 4 sequences of 64
// new tokens 53 and 104, of 128 90 and 104; 16 of 32 90 and 106, of 64 160 and 106;
// 64 of 1000 keys (2 waves) and 16 new tokens 47 and 53, 32 68 and 53.
bool kv8_packed(int N) { return N < 2 * attn47::fwd_box_rows(); }
bool kv8_in_tiles(int num_seqs, int Hq, int Hkv, int N, int d) {
  constexpr double kCtas = 152;
  const long long rows = static_cast<long long>(Hq / Hkv) * N, tile = 2 * attn47::fwd_box_rows();
  const double seqs = num_seqs;
  const double units = kv8_packed(N) ? seqs * Hkv * ((rows + tile - 1) / tile) : seqs * Hq * ((N + tile - 1) / tile);
  const attn47::Kv8Rows pass = attn47::decode_kv8_rows(Hq, Hkv, N, d);
  const double share = d == 128 ? 3 : pass.group <= 16 ? 5 : 3.5;   // passes that take a CTA as long as its part of a wave
  return seqs * Hkv * pass.groups > share * kCtas * std::ceil(units / kCtas);
}

// Both attentions over an 8-bit cache.
attn_status_t attend_kv8(const char* what, bool decode, const void* q, const void* kv_cache, const int32_t* block_table,
                         const int32_t* seq_lens, int num_seqs, int Hq, int Hkv, int N, int d, int block_size,
                         int max_blocks_per_seq, int num_blocks, float scale, void* o, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int passes = 1;
  bool tiles = false;
  if (Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && N > 0) {
    if (static_cast<long long>(Hq / Hkv) * N >= 0x7fffff00LL)
      return fail(ATTN_ERR_UNSUPPORTED, "problem too large for one launch");
    tiles = !decode && kv8_in_tiles(num_seqs, Hq, Hkv, N, d);
    if (!tiles) {
      need = attn47::decode_kv8_workspace_bytes(Hq, Hkv, N, d);
      passes = attn47::decode_kv8_rows(Hq, Hkv, N, d).groups;
      // Tiles too where the passes' blocks are more than their split can count.
      if (passes > 1 && static_cast<__int128>(num_seqs) * Hkv * passes * (static_cast<long long>(max_blocks_per_seq) + 64) >= 0x7fffffff) {
        tiles = true;
        need = 0;
        passes = 1;
      }
    }
  }
  DeviceInfo* dev;
  // Records are counted in 31 bits.
  if (static_cast<long long>(num_blocks) * Hkv >= 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "KV pool too large (num_blocks * Hkv >= 2^31)");
  const attn_status_t st = check_quantised_attention(8, 0, decode, q, kv_cache, block_table, seq_lens, num_seqs, Hq, Hkv,
                                                     N, d, block_size, max_blocks_per_seq, num_blocks, scale, o, lse,
                                                     workspace, workspace_bytes, need, passes, &dev);
  if (st != ATTN_OK || dev == nullptr) return st;
  if (tiles) {
    // The heads of a group in one row of query blocks where N is short.
    const bool packed = kv8_packed(N);
    const int heads = packed ? Hkv : Hq, rows = packed ? Hq / Hkv * N : N;
    const cuuint32_t qbox[3] = {64, static_cast<cuuint32_t>(attn47::fwd_box_rows()), 1};
    const cuuint64_t qdims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows),
                                 static_cast<cuuint64_t>(num_seqs) * heads};
    alignas(64) CUtensorMap tq, blocks;
    attn_status_t enc = encode_bf16(&tq, q, 3, qdims, qbox);
    if (enc == ATTN_OK) enc = encode_kv8(&blocks, kv_cache, static_cast<cuuint64_t>(num_blocks) * Hkv, d);
    if (enc != ATTN_OK) return enc;
    attn47::FwdLaunch f;
    f.tq = &tq;
    f.tk = &blocks;
    f.tv = &blocks;   // (not used)
    f.o = o;
    f.lse = lse;
    f.B = num_seqs;
    f.Hq = heads;
    f.Hkv = Hkv;
    f.N = rows;
    f.d = d;
    f.causal = true;
    f.scale = scale;
    f.sms = dev->sms;
    f.status = dev->status;
    f.timeout_ns = g_timeout_ns;
    f.stream = static_cast<cudaStream_t>(stream);
    f.paged = true;
    f.block_table = block_table;
    f.ctx_lens = seq_lens;
    f.max_blocks = max_blocks_per_seq;
    f.num_blocks = num_blocks;
    f.kv_cache = kv_cache;
    f.q = q;
    f.rows = N;
    return launch_result(attn47::launch_fwd_sm103(f), what);
  }
  attn47::DecKv8Launch a;
  fill_quantised_decode(a, *dev, q, kv_cache, block_table, seq_lens, num_seqs, Hq, Hkv, d, max_blocks_per_seq, num_blocks,
                        scale, o, lse, workspace, stream);
  a.N = N;
  alignas(64) CUtensorMap records;
  const attn_status_t enc = encode_kv8(&records, kv_cache, static_cast<cuuint64_t>(num_blocks) * Hkv, d);
  if (enc != ATTN_OK) return enc;
  a.records = &records;
  return launch_result(attn47::launch_decode_kv8_sm103(a), what);
}

__global__ void selftest_wait_kernel(unsigned int* status, unsigned long long timeout_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    attn47::mbar_init(attn47::smem_addr(&bar), 1);
    abort_flag = 0;
    attn47::fence_mbar_init();
  }
  __syncwarp();
  const attn47::WaitCtl wc{&abort_flag, status, timeout_ns};
  // Nothing arrives on `bar`: the wait must give up after timeout_ns.
  attn47::mbar_wait_warp(attn47::smem_addr(&bar), 0, wc);
}

}  // namespace

extern "C" {

int attn_abi_version(void) { return ATTN47_ABI_VERSION; }

const char* attn_last_error(void) { return g_last_error; }

const char* attn_status_string(attn_status_t s) {
  switch (s) {
    case ATTN_OK: return "ATTN_OK";
    case ATTN_ERR_INVALID_ARG: return "ATTN_ERR_INVALID_ARG";
    case ATTN_ERR_UNSUPPORTED: return "ATTN_ERR_UNSUPPORTED";
    case ATTN_ERR_DEVICE: return "ATTN_ERR_DEVICE";
    case ATTN_ERR_LAUNCH: return "ATTN_ERR_LAUNCH";
    case ATTN_ERR_WORKSPACE: return "ATTN_ERR_WORKSPACE";
  }
  return "ATTN_ERR_UNKNOWN";
}

void attn_set_wait_timeout_ns(unsigned long long ns) { g_timeout_ns = ns < 1000ull ? 1000ull : ns; }

void attn_set_decode_max_ctas(int ctas) { g_decode_max_ctas = ctas > 0 ? ctas : 0; }

void attn_set_decode_early_plan(int on) { g_decode_early_plan.store(on <= 0 ? 0 : on >= 2 ? 2 : 1); }

attn_status_t attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                       int Hq, int Hkv, int N, int d, int causal, float scale, void* stream) {
  if (B < 0 || N < 0 || Hq < 1 || Hkv < 1)
    return fail(ATTN_ERR_INVALID_ARG, "sizes must satisfy B >= 0, N >= 0, Hq >= 1, Hkv >= 1");
  if (Hq % Hkv != 0) return fail(ATTN_ERR_INVALID_ARG, "Hq (%d) is not a multiple of Hkv (%d)", Hq, Hkv);
  if (!finite_positive(scale)) return fail(ATTN_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", d);
  if (B == 0 || N == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if (!q || !k || !v || !o) return fail(ATTN_ERR_INVALID_ARG, "q, k, v and o must be non-null");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o))
    return fail(ATTN_ERR_INVALID_ARG, "q, k, v and o must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  const long long tiles = (static_cast<long long>(N) + 127) / 128;
  if (static_cast<long long>(B) * Hq * tiles > 0x7fffffffLL || static_cast<long long>(B) * Hq > 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "problem too large for one launch");
  DeviceInfo* dev = nullptr;
  attn_status_t st = current_device(&dev);
  if (st != ATTN_OK) return st;
  const size_t qb = static_cast<size_t>(B) * Hq * N * d * 2, kvb = static_cast<size_t>(B) * Hkv * N * d * 2;
  if ((st = check_bufs(*dev, {{q, qb, "q"}, {k, kvb, "k"}, {v, kvb, "v"}, {o, qb, "o"},
                              {lse, static_cast<size_t>(B) * Hq * N * 4, "lse"}})) != ATTN_OK)
    return st;

  const cuuint32_t rows = static_cast<cuuint32_t>(attn47::fwd_box_rows());
  const cuuint32_t box[3] = {64, rows, 1};
  const cuuint64_t dq[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                            static_cast<cuuint64_t>(B) * Hq};
  const cuuint64_t dkv[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                             static_cast<cuuint64_t>(B) * Hkv};
  alignas(64) CUtensorMap tq, tk, tv;
  if ((st = encode_bf16(&tq, q, 3, dq, box)) != ATTN_OK) return st;
  if ((st = encode_bf16(&tk, k, 3, dkv, box)) != ATTN_OK) return st;
  if ((st = encode_bf16(&tv, v, 3, dkv, box)) != ATTN_OK) return st;

  attn47::FwdLaunch a;
  a.tq = &tq;
  a.tk = &tk;
  a.tv = &tv;
  a.o = o;
  a.lse = lse;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.N = N;
  a.d = d;
  a.causal = causal != 0;
  a.scale = scale;
  a.sms = dev->sms;
  a.status = dev->status;
  a.timeout_ns = g_timeout_ns;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_result(attn47::launch_fwd_sm103(a), "attn_fwd");
}

size_t attn_bwd_workspace_size(int B, int Hq, int N) {
  if (B <= 0 || Hq <= 0 || N <= 0) return 0;
  return attn47::bwd_workspace_bytes(B, Hq, N);
}

attn_status_t attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                       const void* dout, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N,
                       int d, int causal, float scale, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (B < 0 || N < 0 || Hq < 1 || Hkv < 1)
    return fail(ATTN_ERR_INVALID_ARG, "sizes must satisfy B >= 0, N >= 0, Hq >= 1, Hkv >= 1");
  if (Hq % Hkv != 0) return fail(ATTN_ERR_INVALID_ARG, "Hq (%d) is not a multiple of Hkv (%d)", Hq, Hkv);
  if (!finite_positive(scale)) return fail(ATTN_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", d);
  if (B == 0 || N == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv)
    return fail(ATTN_ERR_INVALID_ARG, "q, k, v, o, lse, dout, dq, dk and dv must be non-null");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return fail(ATTN_ERR_INVALID_ARG, "q, k, v, o, dout, dq, dk and dv must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return fail(ATTN_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  const size_t need = attn47::bwd_workspace_bytes(B, Hq, N);
  if (!workspace) return fail(ATTN_ERR_INVALID_ARG, "workspace must be non-null");
  if ((reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  if (workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace too small: %zu bytes given, %zu needed", workspace_bytes, need);
  const long long tiles = (static_cast<long long>(N) + 127) / 128;
  if (static_cast<long long>(B) * Hq * tiles > 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "problem too large for one launch");
  DeviceInfo* dev = nullptr;
  attn_status_t st = current_device(&dev);
  if (st != ATTN_OK) return st;
  const size_t qb = static_cast<size_t>(B) * Hq * N * d * 2, kvb = static_cast<size_t>(B) * Hkv * N * d * 2;
  if ((st = check_bufs(*dev, {{q, qb, "q"}, {k, kvb, "k"}, {v, kvb, "v"}, {o, qb, "o"},
                              {lse, static_cast<size_t>(B) * Hq * N * 4, "lse"}, {dout, qb, "dout"},
                              {dq, qb, "dq"}, {dk, kvb, "dk"}, {dv, kvb, "dv"},
                              {workspace, need, "workspace"}})) != ATTN_OK)
    return st;

  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(attn47::bwd_box_rows()), 1};
  const cuuint64_t dq_dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                                 static_cast<cuuint64_t>(B) * Hq};
  const cuuint64_t dkv_dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                                  static_cast<cuuint64_t>(B) * Hkv};
  alignas(64) CUtensorMap tq, tk, tv, tdo;
  if ((st = encode_bf16(&tq, q, 3, dq_dims, box)) != ATTN_OK) return st;
  if ((st = encode_bf16(&tk, k, 3, dkv_dims, box)) != ATTN_OK) return st;
  if ((st = encode_bf16(&tv, v, 3, dkv_dims, box)) != ATTN_OK) return st;
  if ((st = encode_bf16(&tdo, dout, 3, dq_dims, box)) != ATTN_OK) return st;

  attn47::BwdLaunch a;
  a.tq = &tq;
  a.tk = &tk;
  a.tv = &tv;
  a.tdo = &tdo;
  a.o = o;
  a.dout = dout;
  a.lse = lse;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.N = N;
  a.d = d;
  a.causal = causal != 0;
  a.scale = scale;
  a.workspace = static_cast<float*>(workspace);
  a.status = dev->status;
  a.timeout_ns = g_timeout_ns;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_result(attn47::launch_bwd_sm103(a), "attn_bwd");
}

size_t attn_decode_paged_workspace_size(int num_seqs, int Hq, int d, int max_blocks_per_seq) {
  if (num_seqs <= 0 || Hq <= 0 || d <= 0 || max_blocks_per_seq <= 0) return 0;
  return attn47::decode_workspace_bytes(num_seqs, Hq, d, max_blocks_per_seq);
}

attn_status_t attn_decode_paged(const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* block_table, const int32_t* seq_lens, int num_seqs,
                                int Hq, int Hkv, int d, int block_size, int max_blocks_per_seq,
                                int num_blocks, float scale, void* o, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream) {
  attn_status_t st = decode_check_args(q, k_cache, v_cache, block_table, seq_lens, num_seqs, Hq, Hkv,
                                       d, block_size, max_blocks_per_seq, num_blocks, scale, o, lse);
  if (st != ATTN_OK) return st;
  if (num_seqs == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if (!workspace) return fail(ATTN_ERR_INVALID_ARG, "workspace must be non-null");
  if (!aligned16(workspace)) return fail(ATTN_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  const size_t need = attn_decode_paged_workspace_size(num_seqs, Hq, d, max_blocks_per_seq);
  if (workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  const DecodeBytes nb = decode_bytes(num_seqs, Hq, Hkv, d, max_blocks_per_seq, num_blocks);
  const struct {
    const void* p;
    size_t n;
  } others[] = {{q, nb.q}, {k_cache, nb.cache}, {v_cache, nb.cache}, {block_table, nb.table},
                {seq_lens, nb.lens}, {o, nb.o}, {lse, lse ? nb.lse : 0}};
  for (const auto& x : others)
    if (x.n && overlap(workspace, need, x.p, x.n))
      return fail(ATTN_ERR_INVALID_ARG, "workspace overlaps an input or output of the decode");
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != ATTN_OK) return st;
  if ((st = check_bufs(*dev, {{workspace, need, "workspace"}})) != ATTN_OK) return st;
  return decode_launch(*dev, q, k_cache, v_cache, block_table, seq_lens, num_seqs, Hq, Hkv, d,
                       max_blocks_per_seq, num_blocks, scale, o, lse, workspace, stream);
}

attn_status_t attn_decode_paged_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* block_table, const int32_t* seq_lens,
                                        int num_seqs, int Hq, int Hkv, int d, int block_size,
                                        int max_blocks_per_seq, int num_blocks, float scale,
                                        void* o, float* lse, void* stream) {
  // The same argument checks as attn_decode_paged first, so that both calls
  // give the same answer to the same bad arguments; only then the size of
  // the scratch this decode needs against the built-in array.
  attn_status_t st = decode_check_args(q, k_cache, v_cache, block_table, seq_lens, num_seqs, Hq, Hkv,
                                       d, block_size, max_blocks_per_seq, num_blocks, scale, o, lse);
  if (st != ATTN_OK) return st;
  if (num_seqs == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  const size_t need = attn_decode_paged_workspace_size(num_seqs, Hq, d, max_blocks_per_seq);
  if (need > kNoAllocScratchBytes)
    return fail(ATTN_ERR_WORKSPACE,
                "this decode needs %zu bytes of scratch but the built-in array of "
                "attn_decode_paged_noalloc holds %zu; call attn_decode_paged with a workspace",
                need, kNoAllocScratchBytes);
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != ATTN_OK) return st;
  void* scratch = nullptr;
  {
    // One-time set-up per device (this device is current): the host-side
    // name of the array is not a device address, so look the address up.
    std::lock_guard<std::mutex> lock(g_mu);
    if (dev->noalloc_scratch == nullptr) {
      void* addr = nullptr;
      const cudaError_t e = cudaGetSymbolAddress(&addr, g_attn47_noalloc_scratch);
      if (e != cudaSuccess || addr == nullptr)
        return fail(ATTN_ERR_DEVICE, "scratch array address unavailable: %s", cudaGetErrorString(e));
      dev->noalloc_scratch = addr;
    }
    scratch = dev->noalloc_scratch;
  }
  return decode_launch(*dev, q, k_cache, v_cache, block_table, seq_lens, num_seqs, Hq, Hkv, d,
                       max_blocks_per_seq, num_blocks, scale, o, lse, scratch, stream);
}

attn_status_t attn_prefill_paged(const void* q, const void* k_new, const void* v_new,
                                 void* k_cache, void* v_cache, const int32_t* block_table,
                                 const int32_t* ctx_lens, int num_seqs, int Hq, int Hkv, int N,
                                 int d, int block_size, int max_blocks_per_seq, int num_blocks,
                                 float scale, void* o, float* lse, void* stream) {
  if (num_seqs < 0 || N < 0 || Hq < 1 || Hkv < 1 || max_blocks_per_seq < 1 || num_blocks < 1)
    return fail(ATTN_ERR_INVALID_ARG, "sizes must satisfy num_seqs >= 0, N >= 0, Hq, Hkv, "
                "max_blocks_per_seq, num_blocks >= 1");
  if (Hq % Hkv != 0) return fail(ATTN_ERR_INVALID_ARG, "Hq (%d) is not a multiple of Hkv (%d)", Hq, Hkv);
  if (!finite_positive(scale)) return fail(ATTN_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (block_size != 16) return fail(ATTN_ERR_UNSUPPORTED, "block_size %d not supported (16)", block_size);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", d);
  if (static_cast<long long>(max_blocks_per_seq) * block_size >= 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "max_blocks_per_seq too large");
  if (static_cast<long long>(max_blocks_per_seq) * block_size < N)
    return fail(ATTN_ERR_INVALID_ARG, "N (%d) new tokens do not fit in max_blocks_per_seq (%d) blocks",
                N, max_blocks_per_seq);
  if (num_seqs == 0 || N == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if (!q || !k_new || !v_new || !k_cache || !v_cache || !block_table || !ctx_lens || !o)
    return fail(ATTN_ERR_INVALID_ARG, "q, k_new, v_new, caches, block_table, ctx_lens and o must be non-null");
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(o))
    return fail(ATTN_ERR_INVALID_ARG, "q, k_new, v_new, caches and o must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(ctx_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return fail(ATTN_ERR_INVALID_ARG, "block_table, ctx_lens and lse must be 4-byte aligned");
  const long long tiles = (static_cast<long long>(N) + 127) / 128;
  if (static_cast<long long>(num_seqs) * Hq * tiles > 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "problem too large for one launch");
  DeviceInfo* dev = nullptr;
  attn_status_t st = current_device(&dev);
  if (st != ATTN_OK) return st;
  {
    const size_t qb = static_cast<size_t>(num_seqs) * Hq * N * d * 2;
    const size_t kvb = static_cast<size_t>(num_seqs) * Hkv * N * d * 2;
    const size_t cb = static_cast<size_t>(num_blocks) * Hkv * 16 * d * 2;
    if ((st = check_bufs(*dev, {{q, qb, "q"}, {k_new, kvb, "k_new"}, {v_new, kvb, "v_new"},
                                {k_cache, cb, "k_cache"}, {v_cache, cb, "v_cache"},
                                {block_table, static_cast<size_t>(num_seqs) * max_blocks_per_seq * 4,
                                 "block_table"},
                                {ctx_lens, static_cast<size_t>(num_seqs) * 4, "ctx_lens"}, {o, qb, "o"},
                                {lse, static_cast<size_t>(num_seqs) * Hq * N * 4, "lse"}})) != ATTN_OK)
      return st;
  }

  // Q goes through TMA; the kernel gathers the cached K/V blocks itself.
  const cuuint32_t qbox[3] = {64, static_cast<cuuint32_t>(attn47::fwd_box_rows()), 1};
  const cuuint64_t qdims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                               static_cast<cuuint64_t>(num_seqs) * Hq};
  alignas(64) CUtensorMap tq;
  if ((st = encode_bf16(&tq, q, 3, qdims, qbox)) != ATTN_OK) return st;

  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  attn47::AppendLaunch w;
  w.k_new = k_new;
  w.v_new = v_new;
  w.k_cache = k_cache;
  w.v_cache = v_cache;
  w.block_table = block_table;
  w.ctx_lens = ctx_lens;
  w.B = num_seqs;
  w.Hkv = Hkv;
  w.N = N;
  w.d = d;
  w.max_blocks = max_blocks_per_seq;
  w.num_blocks = num_blocks;
  w.sms = dev->sms;
  w.status = dev->status;
  w.stream = s;
  st = launch_result(attn47::launch_kv_append_sm103(w), "attn_prefill_paged (append)");
  if (st != ATTN_OK) return st;

  attn47::FwdLaunch a;
  a.tq = &tq;
  a.tk = &tq;   // unused in paged mode
  a.tv = &tq;
  a.o = o;
  a.lse = lse;
  a.B = num_seqs;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.N = N;
  a.d = d;
  a.causal = true;
  a.scale = scale;
  a.sms = dev->sms;
  a.status = dev->status;
  a.timeout_ns = g_timeout_ns;
  a.stream = s;
  a.paged = true;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.ctx_lens = ctx_lens;
  a.max_blocks = max_blocks_per_seq;
  a.num_blocks = num_blocks;
  return launch_result(attn47::launch_fwd_sm103(a), "attn_prefill_paged (attention)");
}

attn_status_t fused_add_rmsnorm(const void* x, void* residual, const void* weight, void* out,
                                int rows, int hidden, float eps, void* stream) {
  if (rows < 0 || hidden < 8) return fail(ATTN_ERR_INVALID_ARG, "sizes must satisfy rows >= 0, hidden >= 8");
  if (hidden % 8 != 0)
    return fail(ATTN_ERR_UNSUPPORTED, "hidden (%d) must be a multiple of 8 (16-byte rows)", hidden);
  if (!(std::isfinite(eps) && eps >= 0.f)) return fail(ATTN_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (rows == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if (!x || !residual || !weight || !out)
    return fail(ATTN_ERR_INVALID_ARG, "x, residual, weight and out must be non-null");
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(out))
    return fail(ATTN_ERR_INVALID_ARG, "x, residual, weight and out must be 16-byte aligned");
  const size_t bytes = static_cast<size_t>(rows) * hidden * 2;
  if (overlap(residual, bytes, x, bytes) || overlap(residual, bytes, out, bytes) ||
      overlap(out, bytes, x, bytes) || overlap(weight, static_cast<size_t>(hidden) * 2, residual, bytes) ||
      overlap(weight, static_cast<size_t>(hidden) * 2, out, bytes))
    return fail(ATTN_ERR_INVALID_ARG, "x, residual, weight and out must not overlap");
  DeviceInfo* dev = nullptr;
  attn_status_t st = current_device(&dev);
  if (st != ATTN_OK) return st;
  if ((st = check_bufs(*dev, {{x, bytes, "x"}, {residual, bytes, "residual"},
                              {weight, static_cast<size_t>(hidden) * 2, "weight"}, {out, bytes, "out"}})) != ATTN_OK)
    return st;
  attn47::NormLaunch a;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.out = out;
  a.rows = rows;
  a.hidden = hidden;
  a.eps = eps;
  a.sms = dev->sms;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_result(attn47::launch_add_rmsnorm_sm103(a), "fused_add_rmsnorm");
}

attn_status_t fused_swiglu(const void* gate_up, void* out, int rows, int F, void* stream) {
  if (rows < 0 || F < 8) return fail(ATTN_ERR_INVALID_ARG, "sizes must satisfy rows >= 0, F >= 8");
  if (F % 8 != 0) return fail(ATTN_ERR_UNSUPPORTED, "F (%d) must be a multiple of 8 (16-byte rows)", F);
  if (rows == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if (!gate_up || !out) return fail(ATTN_ERR_INVALID_ARG, "gate_up and out must be non-null");
  if (!aligned16(gate_up) || !aligned16(out))
    return fail(ATTN_ERR_INVALID_ARG, "gate_up and out must be 16-byte aligned");
  if (overlap(gate_up, static_cast<size_t>(rows) * F * 4, out, static_cast<size_t>(rows) * F * 2))
    return fail(ATTN_ERR_INVALID_ARG, "gate_up and out must not overlap");
  DeviceInfo* dev = nullptr;
  attn_status_t st = current_device(&dev);
  if (st != ATTN_OK) return st;
  if ((st = check_bufs(*dev, {{gate_up, static_cast<size_t>(rows) * F * 4, "gate_up"},
                              {out, static_cast<size_t>(rows) * F * 2, "out"}})) != ATTN_OK)
    return st;
  attn47::GluLaunch a;
  a.gate_up = gate_up;
  a.out = out;
  a.rows = rows;
  a.F = F;
  a.sms = dev->sms;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_result(attn47::launch_swiglu_sm103(a), "fused_swiglu");
}

attn_status_t swiglu_projection(const void* x, const void* w_gate_up, void* out, int rows, int hidden,
                                int F, void* stream) {
  if (rows < 0 || hidden < 1 || F < 1)
    return fail(ATTN_ERR_INVALID_ARG, "sizes must satisfy rows >= 0, hidden >= 1, F >= 1");
  if (hidden % attn47::swiglu_proj_k_step() != 0)
    return fail(ATTN_ERR_UNSUPPORTED, "hidden (%d) must be a multiple of %d", hidden, attn47::swiglu_proj_k_step());
  if (F % attn47::swiglu_proj_tile_features() != 0)
    return fail(ATTN_ERR_UNSUPPORTED, "F (%d) must be a multiple of %d", F, attn47::swiglu_proj_tile_features());
  if (static_cast<long long>(rows) > 0x7fffffffLL - 128 || 2LL * F > 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "problem too large for one launch");
  if (rows == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if (!x || !w_gate_up || !out) return fail(ATTN_ERR_INVALID_ARG, "x, w_gate_up and out must be non-null");
  if (!aligned16(x) || !aligned16(w_gate_up) || !aligned16(out))
    return fail(ATTN_ERR_INVALID_ARG, "x, w_gate_up and out must be 16-byte aligned");
  const size_t xb = static_cast<size_t>(rows) * hidden * 2;
  const size_t wb = static_cast<size_t>(2) * F * hidden * 2;
  const size_t ob = static_cast<size_t>(rows) * F * 2;
  if (overlap(out, ob, x, xb) || overlap(out, ob, w_gate_up, wb))
    return fail(ATTN_ERR_INVALID_ARG, "out must not overlap x or w_gate_up");
  DeviceInfo* dev = nullptr;
  attn_status_t st = current_device(&dev);
  if (st != ATTN_OK) return st;
  if ((st = check_bufs(*dev, {{x, xb, "x"}, {w_gate_up, wb, "w_gate_up"}, {out, ob, "out"}})) != ATTN_OK)
    return st;
  CUtensorMap tx, tw;
  const cuuint32_t box[2] = {64, 128};
  const cuuint64_t xdims[2] = {static_cast<cuuint64_t>(hidden), static_cast<cuuint64_t>(rows)};
  if ((st = encode_bf16(&tx, x, 2, xdims, box)) != ATTN_OK) return st;
  const cuuint64_t wdims[2] = {static_cast<cuuint64_t>(hidden), static_cast<cuuint64_t>(2) * F};
  if ((st = encode_bf16(&tw, w_gate_up, 2, wdims, box)) != ATTN_OK) return st;
  attn47::SwigluProjLaunch a;
  a.tx = &tx;
  a.tw = &tw;
  a.out = out;
  a.rows = rows;
  a.F = F;
  a.hidden = hidden;
  a.sms = dev->sms;
  a.status = dev->status;
  a.timeout_ns = g_timeout_ns;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_result(attn47::launch_swiglu_proj_sm103(a), "swiglu_projection");
}

size_t ssd_workspace_size(int batch, int L, int H, int N, int chunk) {
  if (batch <= 0 || L <= 0 || H <= 0 || N <= 0 || chunk <= 0) return 0;
  return attn47::ssd_workspace_bytes(batch, L, H, N, chunk);
}

attn_status_t ssd_chunked_fwd(const void* x, const float* dt, const float* A, const void* B,
                              const void* C, const float* h0, void* y, float* h_final, int batch,
                              int L, int H, int G, int P, int N, int chunk, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (batch < 0 || L < 0 || H < 1 || G < 1)
    return fail(ATTN_ERR_INVALID_ARG, "sizes must satisfy batch >= 0, L >= 0, H >= 1, G >= 1");
  if (H % G != 0) return fail(ATTN_ERR_INVALID_ARG, "H (%d) is not a multiple of G (%d)", H, G);
  if (P != attn47::ssd_head_dim()) return fail(ATTN_ERR_UNSUPPORTED, "head dim P = %d not supported (64)", P);
  if (N != 64 && N != 128) return fail(ATTN_ERR_UNSUPPORTED, "state size N = %d not supported (64 or 128)", N);
  if (chunk != 64 && chunk != 128 && chunk != 256)
    return fail(ATTN_ERR_UNSUPPORTED, "chunk = %d not supported (64, 128 or 256)", chunk);
  if (batch == 0 || L == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if (!x || !dt || !A || !B || !C || !y || !h_final || !workspace)
    return fail(ATTN_ERR_INVALID_ARG, "x, dt, A, B, C, y, h_final and workspace must be non-null");
  if (!aligned16(x) || !aligned16(B) || !aligned16(C) || !aligned16(y) || !aligned16(h_final) ||
      !aligned16(workspace) || (h0 && !aligned16(h0)))
    return fail(ATTN_ERR_INVALID_ARG, "x, B, C, y, h0, h_final and workspace must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(dt) & 3u) || (reinterpret_cast<uintptr_t>(A) & 3u))
    return fail(ATTN_ERR_INVALID_ARG, "dt and A must be 4-byte aligned");
  const long long nc = (static_cast<long long>(L) + chunk - 1) / chunk;
  if (static_cast<long long>(batch) * nc * H * (chunk / 64) > 0x7fffffffLL ||
      static_cast<long long>(batch) * nc * H * P > 0x7fffffffLL || static_cast<long long>(L) + chunk > 0x7fffffffLL)
    return fail(ATTN_ERR_UNSUPPORTED, "problem too large for one launch");
  const size_t need = ssd_workspace_size(batch, L, H, N, chunk);
  if (workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  DeviceInfo* dev = nullptr;
  attn_status_t st = current_device(&dev);
  if (st != ATTN_OK) return st;
  {
    const size_t xb = static_cast<size_t>(batch) * L * H * P * 2;
    const size_t bcb = static_cast<size_t>(batch) * L * G * N * 2;
    const size_t hb = static_cast<size_t>(batch) * H * P * N * 4;
    if ((st = check_bufs(*dev, {{x, xb, "x"}, {dt, static_cast<size_t>(batch) * L * H * 4, "dt"},
                                {A, static_cast<size_t>(H) * 4, "A"}, {B, bcb, "B"}, {C, bcb, "C"},
                                {h0, hb, "h0"}, {y, xb, "y"}, {h_final, hb, "h_final"},
                                {workspace, need, "workspace"}})) != ATTN_OK)
      return st;
  }
  attn47::SsdLaunch a;
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.B = B;
  a.C = C;
  a.h0 = h0;
  a.y = y;
  a.h_final = h_final;
  a.workspace = workspace;
  // Tensor maps: x over (P, H, L, batch), B and C over (N, G, L, batch),
  // the bf16 chunk states in the workspace over (N, batch * nc * H * P).
  CUtensorMap tx, tb, tc, ts;
  {
    const cuuint32_t rows = 64;
    const cuuint64_t xdims[4] = {static_cast<cuuint64_t>(P), static_cast<cuuint64_t>(H),
                                 static_cast<cuuint64_t>(L), static_cast<cuuint64_t>(batch)};
    const cuuint64_t xstr[3] = {static_cast<cuuint64_t>(P) * 2, static_cast<cuuint64_t>(H) * P * 2,
                                static_cast<cuuint64_t>(L) * H * P * 2};
    const cuuint32_t xbox[4] = {64, 1, rows, 1};
    if ((st = encode_bf16_strided(&tx, x, 4, xdims, xstr, xbox)) != ATTN_OK) return st;
    const cuuint64_t bdims[4] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(G),
                                 static_cast<cuuint64_t>(L), static_cast<cuuint64_t>(batch)};
    const cuuint64_t bstr[3] = {static_cast<cuuint64_t>(N) * 2, static_cast<cuuint64_t>(G) * N * 2,
                                static_cast<cuuint64_t>(L) * G * N * 2};
    if ((st = encode_bf16_strided(&tb, B, 4, bdims, bstr, xbox)) != ATTN_OK) return st;
    const cuuint32_t cbox[4] = {64, 1, 128, 1};
    if ((st = encode_bf16_strided(&tc, C, 4, bdims, bstr, cbox)) != ATTN_OK) return st;
    const cuuint64_t sdims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(batch * nc * H * P)};
    const cuuint64_t sstr[1] = {static_cast<cuuint64_t>(N) * 2};
    const cuuint32_t sbox[2] = {64, 64};
    const void* states = static_cast<const uint8_t*>(workspace) + attn47::ssd_states_offset(batch, L, H, chunk);
    if ((st = encode_bf16_strided(&ts, states, 2, sdims, sstr, sbox)) != ATTN_OK) return st;
  }
  a.tx = &tx;
  a.tb = &tb;
  a.tc = &tc;
  a.ts = &ts;
  a.batch = batch;
  a.L = L;
  a.H = H;
  a.G = G;
  a.N = N;
  a.chunk = chunk;
  a.status = dev->status;
  a.timeout_ns = g_timeout_ns;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_result(attn47::launch_ssd_sm103(a), "ssd_chunked_fwd");
}

attn_status_t rope_fwd(const attn_heads_t* q, const attn_heads_t* k, const attn_heads_t* q_out,
                       const attn_heads_t* k_out, const attn_rope_t* rope, int B, int N, int d, void* stream) {
  return rope_apply("rope_fwd", q, k, q_out, k_out, rope, B, N, d, false, stream);
}

attn_status_t rope_bwd(const attn_heads_t* dq_out, const attn_heads_t* dk_out, const attn_heads_t* dq,
                       const attn_heads_t* dk, const attn_rope_t* rope, int B, int N, int d, void* stream) {
  return rope_apply("rope_bwd", dq_out, dk_out, dq, dk, rope, B, N, d, true, stream);
}

attn_status_t rope_append_paged(const attn_heads_t* q, const attn_heads_t* k, const attn_heads_t* v,
                                const attn_heads_t* q_out, const attn_rope_t* rope, void* k_cache,
                                void* v_cache, const int32_t* block_table, const int32_t* seq_ids,
                                const int32_t* positions, int T, int num_seqs, int d, int block_size,
                                int max_blocks_per_seq, int num_blocks, void* stream) {
  return rope_append("rope_append_paged", 16, q, k, v, q_out, rope, k_cache, v_cache, nullptr, 0, block_table, seq_ids,
                     positions, T, num_seqs, d, block_size, max_blocks_per_seq, num_blocks, stream);
}

size_t kv4_record_bytes(int d, int group) {
  if ((d != 64 && d != 128) || (group != 32 && group != 64)) return 0;
  return attn47::kv4_record_bytes_of(d, group);
}

attn_status_t rope_append_paged_kv4(const attn_heads_t* q, const attn_heads_t* k, const attn_heads_t* v,
                                    const attn_heads_t* q_out, const attn_rope_t* rope, void* kv_cache,
                                    int group, const int32_t* block_table, const int32_t* seq_ids,
                                    const int32_t* positions, int T, int num_seqs, int d, int block_size,
                                    int max_blocks_per_seq, int num_blocks, void* stream) {
  const attn_status_t st = check_group(group);
  if (st != ATTN_OK) return st;
  return rope_append("rope_append_paged_kv4", 4, q, k, v, q_out, rope, nullptr, nullptr, kv_cache, group, block_table,
                     seq_ids, positions, T, num_seqs, d, block_size, max_blocks_per_seq, num_blocks, stream);
}

attn_status_t kv4_read_paged(const void* kv_cache, int group, const int32_t* block_table,
                             const int32_t* seq_ids, const int32_t* positions, void* k, void* v, int T,
                             int num_seqs, int Hkv, int d, int block_size, int max_blocks_per_seq,
                             int num_blocks, void* stream) {
  const attn_status_t st = check_group(group);
  if (st != ATTN_OK) return st;
  return read_paged("kv4_read_paged", 4, kv_cache, group, block_table, seq_ids, positions, k, v, T, num_seqs, Hkv, d,
                    block_size, max_blocks_per_seq, num_blocks, stream);
}

size_t kv8_record_bytes(int d) { return d == 64 || d == 128 ? attn47::kv8_record_bytes_of(d) : 0; }

attn_status_t kv8_append_paged(const attn_heads_t* q, const attn_heads_t* k, const attn_heads_t* v,
                                    const attn_heads_t* q_out, const attn_rope_t* rope, void* kv_cache,
                                    const int32_t* block_table, const int32_t* seq_ids, const int32_t* positions,
                                    int T, int num_seqs, int d, int block_size, int max_blocks_per_seq,
                                    int num_blocks, void* stream) {
  return rope_append("kv8_append_paged", 8, q, k, v, q_out, rope, nullptr, nullptr, kv_cache, 0, block_table,
                     seq_ids, positions, T, num_seqs, d, block_size, max_blocks_per_seq, num_blocks, stream);
}

attn_status_t kv8_read_paged(const void* kv_cache, const int32_t* block_table, const int32_t* seq_ids,
                             const int32_t* positions, void* k, void* v, int T, int num_seqs, int Hkv, int d,
                             int block_size, int max_blocks_per_seq, int num_blocks, void* stream) {
  return read_paged("kv8_read_paged", 8, kv_cache, 0, block_table, seq_ids, positions, k, v, T, num_seqs, Hkv, d,
                    block_size, max_blocks_per_seq, num_blocks, stream);
}

size_t attn_decode_paged_kv4_workspace_size(int num_seqs, int Hq, int Hkv, int d) {
  if (num_seqs <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv != 0) return 0;
  return attn47::decode_kv4_workspace_bytes(Hq, Hkv, d);
}

attn_status_t attn_decode_paged_kv4(const void* q, const void* kv_cache, const int32_t* block_table,
                                    const int32_t* seq_lens, int num_seqs, int Hq, int Hkv, int d,
                                    int group, int block_size, int max_blocks_per_seq, int num_blocks,
                                    float scale, void* o, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  attn_status_t st = check_group(group);
  if (st != ATTN_OK) return st;
  DeviceInfo* dev;
  const size_t need = Hq > 0 && Hkv > 0 && Hq % Hkv == 0 ? attn47::decode_kv4_workspace_bytes(Hq, Hkv, d) : 0;
  st = check_quantised_attention(4, group, true, q, kv_cache, block_table, seq_lens, num_seqs, Hq, Hkv, 1, d, block_size,
                                 max_blocks_per_seq, num_blocks, scale, o, lse, workspace, workspace_bytes, need, 1,
                                 &dev);
  if (st != ATTN_OK || dev == nullptr) return st;
  attn47::DecKv4Launch a;
  fill_quantised_decode(a, *dev, q, kv_cache, block_table, seq_lens, num_seqs, Hq, Hkv, d, max_blocks_per_seq, num_blocks,
                        scale, o, lse, workspace, stream);
  a.group = group;
  return launch_result(attn47::launch_decode_kv4_sm103(a), "attn_decode_paged_kv4");
}

size_t attn_decode_paged_kv8_workspace_size(int num_seqs, int Hq, int Hkv, int d) {
  if (num_seqs <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv != 0) return 0;
  return attn47::decode_kv8_workspace_bytes(Hq, Hkv, 1, d);
}

attn_status_t attn_decode_paged_kv8(const void* q, const void* kv_cache, const int32_t* block_table,
                                    const int32_t* seq_lens, int num_seqs, int Hq, int Hkv, int d,
                                    int block_size, int max_blocks_per_seq, int num_blocks, float scale,
                                    void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return attend_kv8("attn_decode_paged_kv8", true, q, kv_cache, block_table, seq_lens, num_seqs, Hq, Hkv, 1, d,
                    block_size, max_blocks_per_seq, num_blocks, scale, o, lse, workspace, workspace_bytes, stream);
}

size_t attn_prefill_paged_kv8_workspace_size(int num_seqs, int Hq, int Hkv, int N, int d) {
  if (num_seqs <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || d <= 0 || Hq % Hkv != 0 ||
      static_cast<long long>(Hq / Hkv) * N >= 0x7fffff00LL || kv8_in_tiles(num_seqs, Hq, Hkv, N, d))
    return 0;
  return attn47::decode_kv8_workspace_bytes(Hq, Hkv, N, d);
}

attn_status_t attn_prefill_paged_kv8(const void* q, const void* kv_cache, const int32_t* block_table,
                                     const int32_t* seq_lens, int num_seqs, int Hq, int Hkv, int N, int d,
                                     int block_size, int max_blocks_per_seq, int num_blocks, float scale,
                                     void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return attend_kv8("attn_prefill_paged_kv8", false, q, kv_cache, block_table, seq_lens, num_seqs, Hq, Hkv, N, d,
                    block_size, max_blocks_per_seq, num_blocks, scale, o, lse, workspace, workspace_bytes, stream);
}

attn_status_t attn_get_device_status(void* stream, unsigned int* flags_out) {
  if (!flags_out) return fail(ATTN_ERR_INVALID_ARG, "flags_out must be non-null");
  DeviceInfo* dev = nullptr;
  attn_status_t st = current_device(&dev);
  if (st != ATTN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned int host = 0;
  cudaError_t e = cudaMemcpyAsync(&host, dev->status, sizeof(host), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(dev->status, 0, sizeof(unsigned int), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return fail(ATTN_ERR_DEVICE, "status read failed: %s", cudaGetErrorString(e));
  *flags_out = host;
  g_last_error[0] = '\0';
  return ATTN_OK;
}

}  // extern "C"

namespace {
// One thread per pair of inputs: y = 2^x by the forward softmax's FMA-pipe
// exp2 (ex2_poly2), for testing that function on the device.
__global__ void selftest_exp2_poly_kernel(const float* x, float* y, int n) {
  const long long i = 2LL * (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x);
  if (i >= n) return;
  const bool two = i + 1 < n;
  float r0, r1;
  attn47::f2_unpack(attn47::ex2_poly2(attn47::f2_pack(x[i], two ? x[i + 1] : 0.f)), r0, r1);
  y[i] = r0;
  if (two) y[i + 1] = r1;
}
}  // namespace

extern "C" {

attn_status_t attn_selftest_exp2_poly(const float* x, float* y, int n, void* stream) {
  if (n < 0) return fail(ATTN_ERR_INVALID_ARG, "n must be >= 0");
  if (n == 0) {
    g_last_error[0] = '\0';
    return ATTN_OK;
  }
  if (!x || !y) return fail(ATTN_ERR_INVALID_ARG, "x and y must be non-null");
  if ((reinterpret_cast<uintptr_t>(x) & 3u) || (reinterpret_cast<uintptr_t>(y) & 3u))
    return fail(ATTN_ERR_INVALID_ARG, "x and y must be 4-byte aligned");
  DeviceInfo* dev = nullptr;
  attn_status_t st = current_device(&dev);
  if (st != ATTN_OK) return st;
  const size_t bytes = static_cast<size_t>(n) * 4;
  if ((st = check_bufs(*dev, {{x, bytes, "x"}, {y, bytes, "y"}})) != ATTN_OK) return st;
  const long long pairs = (static_cast<long long>(n) + 1) / 2;
  return launch_result(attn47::launch(false, selftest_exp2_poly_kernel, dim3(static_cast<unsigned>((pairs + 255) / 256)),
                                      dim3(256), 0, static_cast<cudaStream_t>(stream), x, y, n),
                       "attn_selftest_exp2_poly");
}

attn_status_t attn_selftest_wait_timeout(unsigned long long timeout_ns, void* stream,
                                         unsigned int* flags_out) {
  if (!flags_out) return fail(ATTN_ERR_INVALID_ARG, "flags_out must be non-null");
  if (timeout_ns > 10000000000ull) return fail(ATTN_ERR_INVALID_ARG, "timeout above 10 s");
  DeviceInfo* dev = nullptr;
  attn_status_t st = current_device(&dev);
  if (st != ATTN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = launch_result(attn47::launch(false, selftest_wait_kernel, dim3(1), dim3(32), 0, s, dev->status, timeout_ns),
                     "selftest");
  if (st != ATTN_OK) return st;
  return attn_get_device_status(stream, flags_out);
}

}  // extern "C"
