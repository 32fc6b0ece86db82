// Definitions shared by the feed-forward operators (norm.cu, fp8.cu, moe.cu)
// and their host code (api_ffn.cu).
//
// Weight matrices are stored transposed ("rows" are output columns, K runs
// along the input) and cut into cores of 8 rows x 128 bytes of K (128 e4m3
// or 64 16-bit values), 1 KB each, in the order [matrix][row / 64][K block]
// [row / 8 % 8].  A block that walks along K reads one contiguous stream, and a
// K block of 64 rows (or of 16, 32 of them) is one copy; one or two such groups
// are the operand tile of a tensor-core product as they are (a copy of 1 KB for
// each core instead took the copying thread 1000 clocks a tile).  Inside a core,
// the 16-byte
// chunk c of row r lies at chunk c ^ r (the 128-byte swizzle): a warp's 16-byte
// reads of eight rows meet no shared-memory bank twice, and the tensor core
// takes the tile as it is.  Rows and K are padded with zeros.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace effort {

constexpr int kBlk = 128;            // elements that share one scale
constexpr int kCoreBytes = 1024;     // 8 rows x 128 bytes
constexpr float kE4M3Max = 448.0f;
constexpr int kMaxDevices = 64;      // devices whose launch limits are remembered

// element types of activations and outputs (effort_dtype_t)
enum : int { kF32 = 0, kF16 = 1, kBF16 = 2 };
// weight kinds (effort_weight_kind_t)
enum : int { kWF16 = 0, kWBF16 = 1, kWE4M3 = 2 };

__host__ __device__ inline int k_per_block(int wk) { return wk == kWE4M3 ? 128 : 64; }
__host__ __device__ inline int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

__host__ __device__ inline int align4(int x) { return (x + 3) & ~3; }

constexpr int kGroupCores = 8;       // cores that lie together
constexpr int kGroupBytes = kGroupCores * kCoreBytes;
// offset of a core in a matrix of nkb K blocks
__host__ __device__ inline size_t core_at(int core, int kb, int nkb) {
  return ((size_t)(core / kGroupCores) * nkb + kb) * kGroupBytes + (core % kGroupCores) * kCoreBytes;
}

// One stored matrix, or a stack of them.
struct TileMat {
  const uint8_t* data;
  int cores;           // 8-row groups of one matrix, a multiple of kGroupCores
  int nkb;             // K blocks
  size_t stride;       // bytes from one matrix of the stack to the next
};

// Tensor maps (tensor_map.cu).  False where the driver refuses.
// Rows of bytes as {byte, row}: a copy brings 128 bytes of `box` rows in the
// 128-byte swizzle; bytes and rows outside read as zero.
bool map_rows(CUtensorMap* map, const void* data, long long bytes, long long rows, long long stride, int box);

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// element i of an array whose type is known at run time
__device__ __forceinline__ float load_dt(const void* p, int dt, size_t i) {
  if (dt == kF32) return static_cast<const float*>(p)[i];
  if (dt == kF16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_dt(void* p, int dt, size_t i, float v) {
  if (dt == kF32) static_cast<float*>(p)[i] = v;
  else if (dt == kF16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Two e4m3 values as two binary16 values (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t lo16) {
  uint32_t r;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(r) : "r"(lo16));
  return r;
}
__device__ __forceinline__ float e4m3_to_float(uint8_t b) {
  const uint32_t h = e4m3x2_to_half2(b);
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

}  // namespace effort
