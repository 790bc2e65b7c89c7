// FP8 E4M3 quantisation with one FP32 scale per 1 x 128 block (activations)
// or 128 x 128 block (weights); the rule is in fp8.cuh.
//
// Bound by HBM: 2 bytes in, 1 out per element, the scales are 1/32 or 1/4096
// of that.  The block is held in registers between the maximum and the
// codes, so it is read once.  Measured: 8192 x 2048 BF16 by rows 12.4 us (launch
// included; 4.1 TB/s), 64 x 1280 x 2048 by 128 x 128 blocks 93 us (5.4 TB/s of
// the 6.45 of a copy).
#include "fp8.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

template <typename T16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Pack2<T16>::unpack(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));
  return a;
}
__device__ __forceinline__ uint2 quant8(const float (&v)[8], float r) {
  return make_uint2(fp8_quant4(v[0], v[1], v[2], v[3], r), fp8_quant4(v[4], v[5], v[6], v[7], r));
}

// 1 x 128 blocks: 16 lanes of 8 values each hold one block, four blocks at a
// time (64 bytes a lane in flight).  The two divisions of a block cost as much
// as all its other arithmetic when every lane does them, so lane i of the four
// blocks' 16 does those of block i and the others are told.  `rows` counts the
// rows of all batches (they are contiguous).
constexpr int kBlocks = 4;
template <typename T16>
__global__ void __launch_bounds__(kThreads) k_fp8_quant_rows(const T16* __restrict__ v, size_t rows, int K,
                                                             uint8_t* __restrict__ codes, float* __restrict__ scales) {
  griddep_wait();
  griddep_launch_dependents();
  const int KB = fp8_blocks(K);
  const size_t total = rows * size_t(KB);
  const int lane = threadIdx.x & 31, sub = lane & 15;
  const size_t per_cta = kThreads / 16 * kBlocks, stride = size_t(gridDim.x) * per_cta;
  // both halves of a warp take the same number of rounds (the shuffles name all lanes)
  for (size_t b0 = size_t(blockIdx.x) * per_cta + (threadIdx.x >> 5) * 2 * kBlocks; b0 < total; b0 += stride) {
    // the warp's 8 blocks: halves alternate, so that its loads are contiguous
    uint4 u[kBlocks];
    size_t at[kBlocks];
    bool in[kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const size_t b = b0 + 2 * i + (lane >> 4);
      const size_t row = KB == 1 ? b : b / unsigned(KB);
      const int col = int(b - row * KB) * kFp8Block + sub * 8;
      in[i] = b < total && col < K;
      at[i] = row * size_t(K) + col;
      u[i] = in[i] ? __ldg(reinterpret_cast<const uint4*>(v + at[i])) : make_uint4(0, 0, 0, 0);
    }
    float a[kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      float f[8];
      unpack8<T16>(u[i], f);
      a[i] = amax8(f);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a[i] = fmaxf(a[i], __shfl_xor_sync(0xffffffffu, a[i], o));
    }
    const int mine = lane & (kBlocks - 1);
    const Fp8Scale q = fp8_scale(mine == 0 ? a[0] : mine == 1 ? a[1] : mine == 2 ? a[2] : a[3]);
    const size_t bm = b0 + 2 * mine + (lane >> 4);
    if (sub < kBlocks && bm < total) scales[bm] = q.s;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const float r = __shfl_sync(0xffffffffu, q.r, (lane & 16) + i);
      float f[8];
      unpack8<T16>(u[i], f);
      if (in[i]) *reinterpret_cast<uint2*>(codes + at[i]) = quant8(f, r);
    }
  }
}

// 128 x 128 blocks: one thread block each, 16 threads per row, 8 rows per thread.
template <typename T16>
__global__ void __launch_bounds__(kThreads) k_fp8_quant_tiles(const T16* __restrict__ v, int rows, int K,
                                                              uint8_t* __restrict__ codes,
                                                              float* __restrict__ scales) {
  __shared__ float red[kThreads / 32];
  const int KB = fp8_blocks(K), RB = fp8_blocks(rows);
  const unsigned blk = blockIdx.x;
  const unsigned rest = blk / KB;
  const int kb = int(blk - rest * KB);
  const unsigned batch = rest / RB;
  const int rb = int(rest - batch * RB);
  const int col = kb * kFp8Block + (threadIdx.x & 15) * 8;
  const int row0 = rb * kFp8Block + (threadIdx.x >> 4);
  const size_t base = size_t(batch) * rows * K;
  uint4 u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = row0 + 16 * i;
    u[i] = r < rows && col < K ? __ldg(reinterpret_cast<const uint4*>(v + base + size_t(r) * K + col))
                               : make_uint4(0, 0, 0, 0);
  }
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack8<T16>(u[i], f);
    a = fmaxf(a, amax8(f));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) a = fmaxf(a, red[i]);
  const Fp8Scale q = fp8_scale(a);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = row0 + 16 * i;
    if (r < rows && col < K) {
      float f[8];
      unpack8<T16>(u[i], f);
      *reinterpret_cast<uint2*>(codes + base + size_t(r) * K + col) = quant8(f, q.r);
    }
  }
  if (threadIdx.x == 0) scales[blk] = q.s;
}

template <typename T16>
int quantize_t(const void* v, int batch, int rows, int K, int block_rows, uint8_t* codes, float* scales,
               cudaStream_t stream) {
  const T16* p = static_cast<const T16*>(v);
  if (block_rows == 1) {
    const size_t all = size_t(batch) * rows;
    const size_t per = kThreads / 16 * kBlocks;
    const size_t blocks = (all * fp8_blocks(K) + per - 1) / per;
    const size_t most = size_t(num_sms()) * 8 * 8;
    MOE_CHECK_CUDA(launch_pdl(k_fp8_quant_rows<T16>, dim3(unsigned(blocks < most ? blocks : most)), dim3(kThreads), 0,
                              stream, p, all, K, codes, scales));
  } else {
    const size_t blocks = size_t(batch) * fp8_blocks(rows) * fp8_blocks(K);
    MOE_REQUIRE(blocks <= 0x7fffffffu, MOE_ERR_UNSUPPORTED, "moe_fp8_quantize_b128: %zu blocks in one call", blocks);
    k_fp8_quant_tiles<T16><<<unsigned(blocks), kThreads, 0, stream>>>(p, rows, K, codes, scales);
  }
  MOE_CHECK_CUDA(cudaGetLastError());
  return MOE_OK;
}

}  // namespace

int fp8_quantize(const void* v, int batch, int rows, int K, int block_rows, int dtype, uint8_t* codes, float* scales,
                 cudaStream_t stream) {
  if (batch == 0 || rows == 0 || K == 0) return MOE_OK;
  return dtype == MOE_DTYPE_BF16
             ? quantize_t<__nv_bfloat16>(v, batch, rows, K, block_rows, codes, scales, stream)
             : quantize_t<__half>(v, batch, rows, K, block_rows, codes, scales, stream);
}

}  // namespace moe
