// A whole MoE layer on a few tokens (T <= 16) in one cooperative kernel:
// optional pre-MoE RMSNorm, router, top-k, SwiGLU experts, shared expert and
// the weighted sum, with 16-bit experts or FP8 experts (a scale per block of
// 128, fp8.cuh).
//
// A decode step reads every weight once, so it is bound by HBM; the kernel is
// built as one stream of weights with grid barriers where the data demand
// them, and keeps loads in flight across the barriers.
//
//   phase 0  every block: x (normalised) into shared memory, quantised for
//            FP8 experts; its share of the router rows -> logits; arrive at
//            barrier 1; its share of the shared expert's gate/up rows
//   phase 1  (barrier 1) every block selects every token's experts (one warp
//            per token) and lists the distinct experts; the gate/up rows of
//            all of them form one range of 4-feature units that is split
//            evenly over the blocks; h to the workspace
//   phase 2  (barrier 2; FP8: h is quantised, by every block for itself when
//            it is small, else spread over the grid with a barrier 3)
//            each block owns an even share of the output columns and forms
//            them for every expert, so the weighted sum needs no exchange
//            between blocks
// Weights that do not depend on the selection, or on the barrier about to be
// passed, are requested before it: the shared expert's when the kernel starts,
// the first down rows between arriving at barrier 2 and waiting (not before
// arriving: the release would wait for them).
//
// Products run on mma.sync: the weights are the 16-row A operand and the tokens
// the 8-column B operand.  A dot product does not care which k a lane's 16
// bytes are as long as both operands use the same order, so 16 consecutive
// bytes of a weight row are a lane's fragment.  The copies (cp.async, whole
// 128-byte lines) go to a queue of each warp in shared memory: no other warp
// reads it, so there is no block barrier on the way, the queue can be indexed
// at run time, and 2 to 5 units a warp (what x leaves of the 227 KB, 32 KB a unit
// of all warps; 8 took as long) are in flight.  A few tokens leave the tensor core
// idle most of the time; what counts is the stream: tcgen05 would want the weights
// as whole 128-row tiles and its result back from TMEM, for products that already
// fit in a few registers.  (A ring of registers in place of the queue: 44 / 258 /
// 52 / 103 us on the four layers below; a queue of each lane with 64-byte pieces:
// 38 / 171 / 39 / 84.)
//
// Measured (I = 640, k = 10, shared expert, bias; CUDA events, weights not in L2):
//   BF16 T = 1,  H = 2048, E = 512               88.6 MB   29.1 us
//   FP16 T = 16, H = 2560, E = 256, norm, gate    444 MB    116 to 125 us by selection (3.8 of 6.45 TB/s)
//   FP8  T = 1,  H = 2048, E = 512               49.3 MB   26.7 us
//   FP8  T = 8,  H = 2048, E = 512, norm, gate    152 MB   55.9 us
// While weights stream, gate/up runs at 3.4 (FP8, T = 1) to 6 TB/s (T = 16) and
// down, whose rows are short, at 1.5 to 4; at T = 1 a layer with next to no weights
// takes 15 us: x and the norm 2, the router 2, each grid barrier 1.5 to 2, the
// selection 2.5.  The four-launch form of the same BF16 layer takes 41 us at T = 1.
// A fifth of the warps' time goes to instruction fetch, so the loops are kept short:
// unrolled twice, gate/up costs 1 us at T = 1 and down 1 to 8.
//
// Every sum is FP32.  The same call gives the same bits; the order of a token's
// sums depends on the sizes and on how many distinct experts the batch selects
// (how many warps share a group of gate/up units, where the warps' runs of down
// units are cut), so its last bits may change with the other tokens.  The router adds its pieces of
// 32 products (one FP32 sum of the tensor core each: 32 additions, off by at most
// 2^-18 of the terms' magnitudes) in FP64, so the error of a logit does not grow
// with H; x_norm is rounded to 16 bits from a value accurate beyond FP32, since
// the selection depends on it.  For 16-bit weights h is kept as the sum of two 16-bit
// numbers (the tensor core's operand type; hi + lo holds it to 2^-16 of its
// value in BF16, 2^-22 or 2^-25 in FP16, so y carries one 16-bit rounding, not two: one rounded h had
// 1.4 to 1.55 times the error); FP8 experts quantise h from FP32.
#include <cooperative_groups.h>

#include <type_traits>
#include <utility>

#include "fp8.cuh"
#include "route.cuh"

namespace cg = cooperative_groups;

namespace moe {

constexpr int kLayerDecodeMaxT = 16;
constexpr int kLayerDecodeMaxH = 4096;
constexpr int kLayerDecodeMaxTH = 40960;  // T * H: x (and its codes) in shared memory
constexpr int kLayerDecodeMaxI = 8192;
constexpr int kLayerDecodeMaxE = 1024;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSlots = 16;               // selected experts per token
constexpr int kMaxList = kLayerDecodeMaxT * kMaxSlots;
constexpr int kUnitBytes = 16 * 128;        // a row unit
constexpr int kSlotBytes = kWarps * kUnitBytes;
constexpr int kMaxDepth = 5;
// FP8: up to this size every block quantises all of h for itself, into shared
// memory, which saves a grid barrier.
// At T = 1 (13 KB) 27.4 us against 28.8 with the barrier; at T = 2 (26 KB) the two are
// even, so larger h is spread over the grid.
constexpr int kStageBytes = 16 * 1024;
constexpr int kSmemMax = 227 * 1024;

// Byte offsets into the dynamic shared memory (x16 is at 0).
struct Layout {
  int xsc, red, slot, list, tmask, ent, bits, sel_idx, sel_w, gate, dsum, stage, queue;
};

struct Args {
  const void* x;
  int T, H, E, k, I;
  const void* norm_w;     // or null
  float eps;
  const void* gate_w;     // shared-expert gate, or null
  const void* w_router;
  const float* bias;      // or null
  const uint8_t* w_gu;    // routed experts, 16-bit or E4M3
  const uint8_t* w_d;
  const float* sc_gu;     // FP8 scales
  const float* sc_d;
  const uint8_t* sh_gu;   // shared expert, 16-bit, or null
  const uint8_t* sh_d;
  int32_t* topk_idx;      // or null
  float* topk_w;          // or null
  void* y;
  float* logits;          // [T, E]
  void* h;                // [T * k][hi I | lo I] 16-bit, or [T * k, I] FP32 for FP8 experts
  void* h_sh;             // [T][hi I | lo I] 16-bit
  __half* hq;             // FP8, not staged: h's codes as FP16 values in operand order [T * k, I], and their scales
  float* hs;
  int staged;             // FP8: every block keeps h's codes in shared memory
  int depth;              // queue slots per warp, 2 .. kMaxDepth
  // multipliers of div_small for the divisors I/4, k, the grid and the 128-feature blocks of I
  uint32_t by_ui, by_k, by_grid, by_ib;
  Layout at;
};

// v / d by multiplication with floor(2^32 / d) + 1: exact while v * d < 2^32
// (integer division costs a hundred instructions on the way to every barrier).
__host__ __device__ inline uint32_t div_magic(int d) { return d == 1 ? 0u : 0xffffffffu / uint32_t(d) + 1u; }
__device__ __forceinline__ int div_small(int v, uint32_t magic) {
  return magic ? int(__umulhi(uint32_t(v), magic)) : v;  // 0: divisor 1
}
// The even share of block b of n things over the grid: start, and the next block's.
__device__ __forceinline__ int2 share_of(int n, uint32_t by_grid) {
  const int q = div_small(n, by_grid), r = n - q * int(gridDim.x), b = blockIdx.x;
  const int lo = q * b + min(b, r);
  return make_int2(lo, lo + q + (b < r ? 1 : 0));
}

// n: 16 bytes are copied, or 0 and zeros are written
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_n() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_wait(int pending) {  // 1 .. kMaxDepth - 1
  if (pending >= 3) {
    if (pending == 3) cp_async_wait_n<3>(); else cp_async_wait_n<4>();
  } else {
    if (pending == 2) cp_async_wait_n<2>(); else cp_async_wait_n<1>();
  }
}

enum { MMA_BF16, MMA_F16 };
template <typename T16>
struct MmaKind {
  static constexpr int v = std::is_same<T16, __nv_bfloat16>::value ? MMA_BF16 : MMA_F16;
};
template <int KIND>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if (KIND == MMA_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int KIND>
__device__ __forceinline__ void mma_half(float (&d)[4], const uint4& lo, const uint4& hi, const uint4& b) {
  mma<KIND>(d, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
  mma<KIND>(d, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

// Shared memory.  The offsets are computed on the host and read from the
// kernel's constant arguments, so they cost no registers.
struct Smem {
  const Args& a;
  template <typename V>
  static __device__ __forceinline__ V* at(int off) {
    extern __shared__ __align__(128) uint8_t smem[];
    return reinterpret_cast<V*>(smem + off);
  }
  __device__ __forceinline__ uint8_t* x16() const { return at<uint8_t>(0); }             // [T] rows of x16_pitch bytes
  __device__ __forceinline__ float* xsc() const { return at<float>(a.at.xsc); }          // [T, KB] (FP8)
  __device__ __forceinline__ float* red() const { return at<float>(a.at.red); }          // partial results
  __device__ __forceinline__ int8_t* slot() const { return at<int8_t>(a.at.slot); }      // [expert][16 tokens] slot, -1: not selected
  __device__ __forceinline__ int* list() const { return at<int>(a.at.list); }            // distinct experts, ascending
  __device__ __forceinline__ uint32_t* tmask() const { return at<uint32_t>(a.at.tmask); }  // [expert] tokens that selected it
  __device__ __forceinline__ uint8_t* ent() const { return at<uint8_t>(a.at.ent); }      // [expert][16] those: token | slot << 4
  __device__ __forceinline__ uint32_t* bits() const { return at<uint32_t>(a.at.bits); }  // selected experts, one bit each
  __device__ __forceinline__ int* sel_idx() const { return at<int>(a.at.sel_idx); }      // [T][16]
  __device__ __forceinline__ float* sel_w() const { return at<float>(a.at.sel_w); }
  __device__ __forceinline__ float* gate() const { return at<float>(a.at.gate); }        // [T] factor of the shared expert
  __device__ __forceinline__ double* dsum() const { return at<double>(a.at.dsum); }      // [16] per warp
  __device__ __forceinline__ uint8_t* stage() const { return at<uint8_t>(a.at.stage); }  // h rows (and FP8 scales), when they fit
  __device__ __forceinline__ uint8_t* queue() const { return at<uint8_t>(a.at.queue); }  // depth slots
};
constexpr int kRedBytes = 4 * kWarps * 128 * 4;
__host__ __device__ inline int x16_pitch(int H) { return 2 * H + 64; }  // rows 64 bytes apart modulo 128: no bank conflict
__host__ __device__ inline size_t a16(size_t v) { return (v + 15) / 16 * 16; }
inline Layout layout_of(int T, int H, bool f8, size_t stage) {
  Layout l{};
  size_t p = a16(size_t(T) * x16_pitch(H));
  auto take = [&](size_t n) {
    const size_t r = p;
    p += a16(n);
    return int(r);
  };
  l.xsc = take(f8 ? size_t(T) * fp8_blocks(H) * 4 : 0);
  l.red = take(kRedBytes);
  l.slot = take(size_t(kMaxList) * 16);
  l.list = take(size_t(kMaxList) * 4);
  l.tmask = take(size_t(kMaxList) * 4);
  l.ent = take(size_t(kMaxList) * 16);
  l.bits = take(32 * 4);
  l.sel_idx = take(kLayerDecodeMaxT * kMaxSlots * 4);
  l.sel_w = take(kLayerDecodeMaxT * kMaxSlots * 4);
  l.gate = take(16 * 4);
  l.dsum = take(16 * 8);
  l.stage = take(stage);
  l.queue = int((p + 127) / 128 * 128);  // row units keep the 128-byte lines of their swizzle
  return l;
}
// FP8: the codes of h and their scales, when every block keeps them itself.
__host__ __device__ inline int stage_scales(int T, int k, int I) { return T * k * I * 2; }
inline size_t stage_bytes(int T, int k, int I) { return size_t(stage_scales(T, k, I)) + size_t(T) * k * fp8_blocks(I) * 4; }

// E4M3 operands run on the FP16 tensor core: every E4M3 value is an FP16 value
// and the products are exact in FP32.  (mma.sync with E4M3 operands is carried
// out that way too, converting both operands on every use: about 8 instructions
// where an FP16 one takes 1.)  The weights are converted as they leave the queue;
// the tokens' codes are kept as FP16 values in the order that the 16 weight
// bytes of a lane ask for: in each 64 features, feature 16 t + 8 p + i lies at
// 32 p + 8 t + i, so a lane's pieces p of all four t are 64 consecutive bytes.
__device__ __forceinline__ int operand_order(int k) {
  return (k & ~63) | ((k & 8) << 2) | ((k >> 1) & 24) | (k & 7);
}
__device__ __forceinline__ uint2 e4m3x4_to_f16(uint32_t v) {
  uint2 r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(v));
  return r;
}
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t lo, uint32_t hi, uint32_t b0, uint32_t b1) {
  const uint2 l = e4m3x4_to_f16(lo), h = e4m3x4_to_f16(hi);
  mma<MMA_F16>(d, l.x, h.x, l.y, h.y, b0, b1);
}
// One unit's products in two chains: b are the token's four pieces.
template <int KIND>
__device__ __forceinline__ void unit_e4m3(float (&v)[4], const uint4& lo0, const uint4& hi0, const uint4& lo1,
                                          const uint4& hi1, const uint4 (&b)[4]) {
  static_assert(KIND == MMA_F16, "E4M3 values are held as FP16");
  float p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = p[i] = 0.0f;
  mma_e4m3(v, lo0.x, hi0.x, b[0].x, b[0].y);
  mma_e4m3(p, lo1.x, hi1.x, b[2].x, b[2].y);
  mma_e4m3(v, lo0.y, hi0.y, b[0].z, b[0].w);
  mma_e4m3(p, lo1.y, hi1.y, b[2].z, b[2].w);
  mma_e4m3(v, lo0.z, hi0.z, b[1].x, b[1].y);
  mma_e4m3(p, lo1.z, hi1.z, b[3].x, b[3].y);
  mma_e4m3(v, lo0.w, hi0.w, b[1].z, b[1].w);
  mma_e4m3(p, lo1.w, hi1.w, b[3].z, b[3].w);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] += p[i];
}

// Lanes that share one result of a reduction over n results: a power of two,
// at most 16, so that the block's threads cover the results.
__device__ __forceinline__ int split_of(int n) {
  int p = 1;
  while (p < 16 && p * 2 * n <= kThreads) p *= 2;
  return p;
}

// ---------------------------------------------------------------------------
// phase 0
// ---------------------------------------------------------------------------
// Whether FP32 v lies within 5 of its own steps of a rounding border of T16 (or
// where FP16 is subnormal): there the FP64 value decides.  The FP32 product
// below takes four roundings, so it is off by at most 4 of its steps.
template <typename T16>
__device__ __forceinline__ bool near_border(float v) {
  const uint32_t u = __float_as_uint(v);
  if constexpr (std::is_same<T16, __nv_bfloat16>::value) return ((u & 0xffffu) - 0x7ffbu) <= 10u;
  return ((u & 0x1fffu) - 0x0ffbu) <= 10u || (u & 0x7fffffffu) < 0x38800000u;
}
// far: r itself left FP32's normal range (tokens of about 2^126 and more, or with a
// norm below 2^-128: both need BF16).
template <typename T16>
__device__ __forceinline__ uint32_t norm_pair(float2 f, float2 w, float r, double rd, bool far) {
  const float a = f.x * r * (1.0f + w.x), b = f.y * r * (1.0f + w.y);
  if (far || near_border<T16>(a) || near_border<T16>(b)) {
    const double ad = double(f.x) * rd * (1.0 + double(w.x)), bd = double(f.y) * rd * (1.0 + double(w.y));
    T16 o[2];
    if constexpr (std::is_same<T16, __nv_bfloat16>::value) {
      o[0] = __double2bfloat16(ad);
      o[1] = __double2bfloat16(bd);
    } else {
      o[0] = __double2half(ad);
      o[1] = __double2half(bd);
    }
    return uint32_t(*reinterpret_cast<uint16_t*>(&o[0])) | (uint32_t(*reinterpret_cast<uint16_t*>(&o[1])) << 16);
  }
  return Pack2<T16>::pack(a, b);
}

// Requests x [T, H] and the norm and gate vectors into shared memory (one
// group); the vectors take the two halves of s.red() until the products start.
__device__ __forceinline__ uint8_t* norm_w_of(const Smem& s) { return reinterpret_cast<uint8_t*>(s.red()); }
__device__ __forceinline__ uint8_t* gate_w_of(const Smem& s) { return reinterpret_cast<uint8_t*>(s.red()) + kRedBytes / 2; }
static_assert(kLayerDecodeMaxH * 2 <= kRedBytes / 2, "a norm or gate vector must fit in half of red");
__device__ void fetch_x(const Args& a, const Smem& s) {
  const int nv = a.H / 8;
  const uint8_t* x = static_cast<const uint8_t*>(a.x);
#pragma unroll 1
  for (int c = threadIdx.x; c < nv; c += kThreads) {
#pragma unroll 4
    for (int t = 0; t < a.T; ++t)
      cp_async_16(smem_u32(s.x16() + size_t(t) * x16_pitch(a.H) + c * 16), x + (size_t(t) * nv + c) * 16, 16);
    if (a.norm_w) cp_async_16(smem_u32(norm_w_of(s) + c * 16), static_cast<const uint8_t*>(a.norm_w) + c * 16, 16);
    if (a.gate_w) cp_async_16(smem_u32(gate_w_of(s) + c * 16), static_cast<const uint8_t*>(a.gate_w) + c * 16, 16);
  }
  cp_async_commit();
}

// RMSNorm of the rows in place: 16 / T' warps per token (T' the power of two at
// or above T) add the squares, then every thread scales one chunk of columns of
// every token.
constexpr float kSquareMin = 7.8886090522101181e-31f;  // 2^-100
template <typename T16>
__device__ void norm_x(const Args& a, const Smem& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int lg = 4;
  while ((a.T << lg) > kWarps) --lg;
  const int t = warp >> lg;
  const int nv = a.H / 8;
  double ss4[4] = {0.0, 0.0, 0.0, 0.0};  // short chains
  if (t < a.T) {
    float lo = 0.0f;
    const uint4* xr = reinterpret_cast<const uint4*>(s.x16() + size_t(t) * x16_pitch(a.H));
#pragma unroll 4
    for (int c = (warp & ((1 << lg) - 1)) * 32 + lane; c < nv; c += 32 << lg) {
      const uint4 v = xr[c];
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      // A square of at least 2^-126 is exact in FP32 (16 bits at most), and a smaller one beside
      // a sum of 2^-100 or more is off by 2^-50 of it; the sum is taken with its rounding error.
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = Pack2<T16>::unpack(u[j]);
        const float p0 = f.x * f.x, p1 = f.y * f.y;
        const float big = fmaxf(p0, p1), sum = __fadd_rn(p0, p1);
        if (sum >= kSquareMin && sum < INFINITY) {
          lo += __fsub_rn(fminf(p0, p1), __fsub_rn(sum, big));
          ss4[j] += double(sum);
        } else {  // squares rounded or lost in FP32, beyond it, or not finite
          ss4[j] += double(f.x) * double(f.x) + double(f.y) * double(f.y);
        }
      }
    }
    ss4[0] += double(lo);
  }
  double ss = (ss4[0] + ss4[1]) + (ss4[2] + ss4[3]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) s.dsum()[warp] = ss;
  __syncthreads();
  if (threadIdx.x < a.T) {
    double tot = 0.0;
    for (int i = 0; i < (1 << lg); ++i) tot += s.dsum()[(threadIdx.x << lg) + i];
    // FP32 reciprocal square root and two Newton steps in FP64: good to 1e-13
    const double v = tot * (1.0 / double(a.H)) + double(a.eps);
    const float v32 = float(v);
    double rd = double(rsqrtf(v32));
    rd *= 1.5 - 0.5 * v * rd * rd;
    rd *= 1.5 - 0.5 * v * rd * rd;
    if (!(v32 > FLT_MIN && v32 < INFINITY)) rd = 1.0 / sqrt(v);
    reinterpret_cast<double*>(s.sel_idx())[threadIdx.x] = rd;  // the selection's space is still free
  }
  __syncthreads();
  // (token, chunk) pairs over all threads
  int i = 0, c = threadIdx.x;
#pragma unroll 1
  for (;; c += kThreads) {
    for (; c >= nv; c -= nv) ++i;
    if (i >= a.T) break;
    const double rd = reinterpret_cast<const double*>(s.sel_idx())[i];
    const float r = float(rd);
    const bool far = !(r >= FLT_MIN && r < INFINITY);
    uint4* at = reinterpret_cast<uint4*>(s.x16() + size_t(i) * x16_pitch(a.H)) + c;
    const uint4 v = *at, w = reinterpret_cast<const uint4*>(norm_w_of(s))[c];
    const uint32_t u[4] = {v.x, v.y, v.z, v.w}, g[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = norm_pair<T16>(Pack2<T16>::unpack(u[j]), Pack2<T16>::unpack(g[j]), r, rd, far);
    *at = make_uint4(o[0], o[1], o[2], o[3]);
  }
  __syncthreads();
}

// The x rows in shared memory become their E4M3 codes (as FP16 values, in operand
// order) and scales: half a warp per block, whose lanes have all read before any
// writes (the maximum needs them).
template <typename T16>
__device__ void quant_x(const Args& a, const Smem& s) {
  const int KB = fp8_blocks(a.H), n = a.T * KB;
  const int sub = threadIdx.x & 15;
  for (int b0 = (threadIdx.x >> 5) * 2; b0 < n; b0 += kThreads / 16) {
    const int b = b0 + ((threadIdx.x >> 4) & 1);
    int t = 0, kb = b;
    for (; kb >= KB; kb -= KB) ++t;
    const int col = kb * kFp8Block + sub * 8;
    const bool in = b < n && col < a.H;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in) v = *reinterpret_cast<const uint4*>(s.x16() + size_t(t) * x16_pitch(a.H) + col * 2);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    float f[8], m = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = Pack2<T16>::unpack(u[j]);
      f[2 * j] = p.x;
      f[2 * j + 1] = p.y;
      m = fmaxf(m, fmaxf(fabsf(p.x), fabsf(p.y)));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const Fp8Scale q = fp8_scale(m);
    if (in) {
      const uint2 c0 = e4m3x4_to_f16(fp8_quant4(f[0], f[1], f[2], f[3], q.r));
      const uint2 c1 = e4m3x4_to_f16(fp8_quant4(f[4], f[5], f[6], f[7], q.r));
      *reinterpret_cast<uint4*>(s.x16() + size_t(t) * x16_pitch(a.H) + operand_order(col) * 2) =
          make_uint4(c0.x, c0.y, c1.x, c1.y);
    }
    if (b < n && sub == 0) s.xsc()[t * KB + kb] = q.s;
  }
  __syncthreads();
}

// x[t] . w over one 8-value chunk, FP32
template <typename T16>
__device__ __forceinline__ float dot8(const uint4& xv, const float2 (&w)[4]) {
  const uint32_t u[4] = {xv.x, xv.y, xv.z, xv.w};
  float p = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = Pack2<T16>::unpack(u[j]);
    p = fmaf(f.x, w[j].x, p);
    p = fmaf(f.y, w[j].y, p);
  }
  return p;
}

// This block's router rows blockIdx + n * grid, n = 0..7 (which covers E <= 1024
// on 128 or more SMs; more rounds otherwise): the rows are the 8-column operand,
// the tokens the 16-row one.  A warp takes every 16th piece of 32 features, each
// piece's products are summed by the tensor core in FP32 and added in FP64.  The
// first rows are requested before x is read.
constexpr int kRouterPieces = kLayerDecodeMaxH / 32 / kWarps;
template <typename T16>
__device__ __forceinline__ void router_fetch(const Args& a, int e0, uint4 (&v)[kRouterPieces]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = e0 + (lane >> 2) * gridDim.x;
  const uint8_t* wr = static_cast<const uint8_t*>(a.w_router) + size_t(e < a.E ? e : 0) * a.H * 2 + (lane & 3) * 16;
#pragma unroll
  for (int i = 0; i < kRouterPieces; ++i) {
    const int c = warp + kWarps * i;
    v[i] = e < a.E && c * 32 < a.H ? __ldg(reinterpret_cast<const uint4*>(wr + c * 64)) : make_uint4(0, 0, 0, 0);
  }
}
template <typename T16>
__device__ void router(const Args& a, const Smem& s, uint4 (&v)[kRouterPieces]) {
  constexpr int KIND = MmaKind<T16>::v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, tig = lane & 3;
  double* part = reinterpret_cast<double*>(s.red());  // [16 warps][16 tokens][8 rows]
  static_assert(kWarps * 16 * 8 * 8 <= kRedBytes, "router partial sums must fit in red");
  const uint8_t* x0 = s.x16() + size_t(min(g, a.T - 1)) * x16_pitch(a.H) + tig * 16;
  const uint8_t* x1 = s.x16() + size_t(min(g + 8, a.T - 1)) * x16_pitch(a.H) + tig * 16;
#pragma unroll 1
  for (int e0 = blockIdx.x; e0 < a.E; e0 += gridDim.x * 8) {
    if (e0 != blockIdx.x) router_fetch<T16>(a, e0, v);
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kRouterPieces; ++i) {
      const int c = warp + kWarps * i;
      if (c * 32 < a.H) {
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma_half<KIND>(d, *reinterpret_cast<const uint4*>(x0 + c * 64), *reinterpret_cast<const uint4*>(x1 + c * 64), v[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += double(d[j]);
      }
    }
    double* o = part + warp * 128 + 2 * tig;
    o[g * 8] = acc[0];
    o[g * 8 + 1] = acc[1];
    o[(g + 8) * 8] = acc[2];
    o[(g + 8) * 8 + 1] = acc[3];
    __syncthreads();
    // four threads per (token, row), each four warps' parts
    const int item = threadIdx.x >> 2, t = item >> 3, ee = e0 + (item & 7) * int(gridDim.x);
    const double* p = part + (threadIdx.x & 3) * 4 * 128 + item;
    double l = (p[0] + p[128]) + (p[256] + p[384]);
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if ((threadIdx.x & 3) == 0 && t < a.T && ee < a.E)
      a.logits[size_t(t) * a.E + ee] = float(l + (a.bias ? double(__ldg(a.bias + ee)) : 0.0));
    __syncthreads();
  }
}

// The shared expert's factor of token `warp`.
template <typename T16>
__device__ void shared_gate_value(const Args& a, const Smem& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp >= a.T) return;
  float acc = 0.0f;
  if (a.gate_w)
#pragma unroll 2
    for (int c = lane; c < a.H / 8; c += 32) {
      const uint4 v = reinterpret_cast<const uint4*>(gate_w_of(s))[c];
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      float2 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = Pack2<T16>::unpack(u[j]);
      acc += dot8<T16>(*reinterpret_cast<const uint4*>(s.x16() + size_t(warp) * x16_pitch(a.H) + c * 16), w);
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) s.gate()[warp] = a.gate_w ? 1.0f / (1.0f + __expf(-acc)) : 1.0f;
}

// ---------------------------------------------------------------------------
// Selection of one token by one warp: like topk_token, but first the k-th
// largest of the 32 lanes' maxima bounds the k-th largest logit from below, the
// few logits at or above that bound are gathered, and their ranks counted with
// shuffles (about 600 cycles at E = 512 against 2500 for k rounds of two warp
// reductions).  More than 32 at the bound (ties): the rounds.
// ---------------------------------------------------------------------------
// The rounds, out of line: the way there is rare, and code that is stepped over has
// to be fetched.
__device__ __noinline__ void select_rounds(const float* row, int E, int k, int lane, int* idx_out, float* w_out) {
  topk_token<32>(row, E, k, k, lane, idx_out, w_out, nullptr);
}
template <int NV>
__device__ void select_token(const float* row, int E, int k, int lane, int* idx_out, float* w_out, uint32_t* buf) {
  uint32_t key[NV], best = 0;
  float v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = __ldcg(row + min(lane + 32 * i, E - 1));  // all in flight at once
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float x = (v[i] != v[i]) ? -FLT_MAX : v[i];
    key[i] = lane + 32 * i < E ? order_key(x) : 0u;
    best = max(best, key[i]);
  }
  int rank = 0;  // of this lane's maximum among the 32
#pragma unroll 8
  for (int o = 1; o < 32; ++o) {
    const uint32_t other = __shfl_sync(0xffffffffu, best, (lane + o) & 31);
    rank += other > best || (other == best && ((lane + o) & 31) < lane) ? 1 : 0;
  }
  const uint32_t at_k = __ballot_sync(0xffffffffu, rank == k - 1);
  const uint32_t bound = max(1u, __shfl_sync(0xffffffffu, best, __ffs(at_k) - 1));
  int n = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = key[i] >= bound;
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    const int at = n + __popc(m & ((1u << lane) - 1u));
    if (in && at < 32) {
      buf[at] = key[i];
      buf[32 + at] = uint32_t(lane + 32 * i);
    }
    n += __popc(m);
  }
  __syncwarp();
  if (n > 32) {
    select_rounds(row, E, k, lane, idx_out, w_out);
    return;
  }
  const uint32_t my = lane < n ? buf[lane] : 0u;
  const uint32_t ix = lane < n ? buf[32 + lane] : 0xffffffffu;
  rank = 0;
#pragma unroll 8
  for (int o = 1; o < 32; ++o) {
    const uint32_t ok = __shfl_sync(0xffffffffu, my, (lane + o) & 31), oi = __shfl_sync(0xffffffffu, ix, (lane + o) & 31);
    rank += ok > my || (ok == my && oi < ix) ? 1 : 0;
  }
  const uint32_t first = __ballot_sync(0xffffffffu, lane < n && rank == 0);
  const float top = key_value(__shfl_sync(0xffffffffu, my, __ffs(first) - 1));
  const float p = lane < n && rank < k ? __expf(key_value(my) - top) : 0.0f;
  // the sum in rank order, as topk_token's lanes hold it
  if (lane < n && rank < k) {
    idx_out[rank] = int(ix);
    w_out[rank] = p;
  }
  __syncwarp();
  float z = lane < k ? w_out[lane] : 0.0f;
  const float mine = z;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  if (lane < k) w_out[lane] = mine * (1.0f / z);
}

// ---------------------------------------------------------------------------
// A warp's queue of row units.  A unit is 16 rows x 128 bytes of a weight
// matrix, copied 4 whole 128-byte lines per instruction (8 lines of 64 bytes
// took the load unit twice as long: it would bound the stream).  16-byte chunk
// c of row r lies at chunk c ^ 4 (r & 1), so that the fragment reads, lane (g,
// tig) taking chunks tig and 4 + tig of rows g and g + 8, meet no bank conflict.
// A slot is written again only after the products that read it: they are
// warp-wide instructions.
// ---------------------------------------------------------------------------
struct Unit {
  uint4 lo0, hi0, lo1, hi1;
};
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
  return v;
}
struct Queue {
  uint32_t front, back;  // slots 0 .. nf - 1 lie in one area, the others in another (this warp's part)
  uint32_t wr, rd;       // this lane's offsets for copying (row lane / 8) and for reading (row g)
  int nf, depth, in, out;
  // `dead` bytes at `area` (shared memory that the phase has no other use for) come before the queue's own slots
  __device__ Queue(const Smem& s, int own, uint8_t* area, int dead) {
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    nf = min(dead / kSlotBytes, kMaxDepth - own);
    front = smem_u32(area) + warp * kUnitBytes;
    back = smem_u32(s.queue()) + warp * kUnitBytes - nf * kSlotBytes;
    wr = (lane >> 3) * 128 + ((lane & 7) ^ (((lane >> 3) & 1) << 2)) * 16;
    rd = (lane >> 2) * 128 + ((lane & 3) ^ (((lane >> 2) & 1) << 2)) * 16;
    depth = own + nf;
    in = out = 0;
  }
  __device__ __forceinline__ uint32_t at(int slot) const { return (slot < nf ? front : back) + slot * kSlotBytes; }
  // rows lane / 8 + 4 i of the unit, this lane's chunk of each
  __device__ __forceinline__ void push(const uint8_t* r0, const uint8_t* r1, const uint8_t* r2, const uint8_t* r3,
                                       uint32_t n0, uint32_t n1, uint32_t n2, uint32_t n3) {
    const uint32_t d = at(in) + wr;
    cp_async_16(d, r0, n0);
    cp_async_16(d + 512, r1, n1);
    cp_async_16(d + 1024, r2, n2);
    cp_async_16(d + 1536, r3, n3);
  }
  __device__ __forceinline__ void commit() {  // also for an empty slot: the waits count groups
    cp_async_commit();
    in = in + 1 == depth ? 0 : in + 1;
  }
  __device__ __forceinline__ Unit pop() {
    cp_async_wait(depth - 1);
    __syncwarp();
    const uint32_t d = at(out) + rd;
    Unit u;
    u.lo0 = lds128(d);
    u.hi0 = lds128(d + 1024);
    u.lo1 = lds128(d ^ 64);
    u.hi1 = lds128((d ^ 64) + 1024);
    out = out + 1 == depth ? 0 : out + 1;
    return u;
  }
  // a stream ends with depth - 1 empty groups that nobody takes
  __device__ __forceinline__ void reset() { out = in; }
};

// ---------------------------------------------------------------------------
// gate/up rows of units [u0, u1) (4 features each): SHARED, the shared expert
// for every token; else the listed experts for the tokens that selected them.
// Groups of two units are 8 gate rows (g) and the matching 8 up rows (g + 8)
// of an A operand, so gate and up of a feature meet in one lane.
//
// The warps take groups in rounds.  While 16 or more are left each warp takes
// a whole one and nothing is exchanged.  The rest are taken in rounds of a
// power of two, 16 / that many warps sharing the K units of a group, and their
// partial results are added once, at the end of the phase (a reduction and two
// barriers after every few groups, as it was before, held FP8 experts to 4.1
// TB/s where this reaches 5).
// ---------------------------------------------------------------------------
template <typename T16, bool F8, int NT, bool SHARED>
struct GateUp {
  static constexpr int KIND = F8 ? MMA_F16 : MmaKind<T16>::v;
  static constexpr int ES = F8 ? 1 : 2;
  static constexpr int STAGES = 4 / NT;  // shared rounds that fit in red
  const Args& a;
  const Smem& s;
  const uint8_t* w;
  Queue& q;
  int u0, u1, groups, row_bytes, KU, UI, g, tig, warp;
  // position: first group of the round, log2 of the warps that share a group (16 groups a round at 0)
  struct Round {
    int first, lg, shared;  // shared: rounds with lg > 0 so far
  };
  // issue position, and the lane's row pointers
  Round ir;
  int iu;
  const uint8_t *pa, *pb;  // gate rows lane / 8 and lane / 8 + 4: the group's first and second unit
  uint32_t n_b;            // a group has its first unit, not always its second
  size_t up;               // from a gate row to its up row

  __device__ GateUp(const Args& a_, const Smem& s_, const uint8_t* w_, Queue& q_, int u0_, int u1_)
      : a(a_), s(s_), w(w_), q(q_), u0(u0_), u1(u1_) {
    const int lane = threadIdx.x & 31;
    warp = threadIdx.x >> 5;
    g = lane >> 2;
    tig = lane & 3;
    row_bytes = a.H * ES;
    KU = (row_bytes + 127) / 128;
    up = size_t(a.I) * row_bytes;
    UI = a.I / 4;
    groups = (u1 - u0 + 1) / 2;
    ir = {0, 0, 0};
    width_of(ir);
    enter();
  }
  // The round's width: 16 groups, or the largest power of two that is left (the
  // smallest that holds the rest in the last shared round).
  __device__ __forceinline__ void width_of(Round& r) const {
    const int left = groups - r.first;
    r.lg = 0;
    if (left > 0 && left < kWarps) {
      int lc = 31 - __clz(left);
      if (r.shared == STAGES - 1 && (1 << lc) < left) ++lc;
      r.lg = 4 - lc;
    }
  }
  __device__ __forceinline__ void next(Round& r) const {
    r.first += kWarps >> r.lg;
    r.shared += r.lg > 0 ? 1 : 0;
    width_of(r);
  }
  __device__ __forceinline__ int group_of(const Round& r) const { return r.first + (warp >> r.lg); }
  __device__ __forceinline__ int k0_of(const Round& r) const { return warp & ((1 << r.lg) - 1); }
  // The next round of the issue position in which this warp has a unit.
  __device__ __forceinline__ void enter() {
    while (ir.first < groups && (group_of(ir) >= groups || k0_of(ir) >= KU)) next(ir);
    if (ir.first < groups) {
      iu = k0_of(ir);
      const int u = u0 + 2 * group_of(ir);
      n_b = u + 1 < u1 ? 16 : 0;
      pa = row_of(u);
      pb = n_b ? row_of(u + 1) : pa;
    }
  }
  __device__ __forceinline__ const uint8_t* row_of(int u) const {
    const int lane = threadIdx.x & 31;
    const int ei = div_small(u, a.by_ui), f = (u - ei * UI) * 4 + (lane >> 3);
    return w + (size_t(SHARED ? 0 : s.list()[ei]) * 2 * a.I + f) * row_bytes + (lane & 7) * 16;
  }
  // FP8 weight scales of unit u's rows: [K block] for gate, fp8_blocks(I) rows later
  // for up.  They are read as they are needed, one K unit's while the next waits in
  // the queue (a table of the block's scales in shared memory, filled before the
  // weights are asked for, took as long: 57.7 against 58.9 us at T = 8).
  __device__ __forceinline__ const float* scales_of(int u) const {
    const int IB = fp8_blocks(a.I), ei = div_small(u, a.by_ui);
    return a.sc_gu + (size_t(s.list()[ei]) * 2 * IB + ((u - ei * UI) >> 5)) * fp8_blocks(a.H);
  }
  __device__ __forceinline__ void issue() {
    if (ir.first < groups) {
      // only FP8 rows can end inside a unit
      const bool in = !F8 || iu * 128 + int(threadIdx.x & 7) * 16 < row_bytes;
      const uint32_t na = in ? 16 : 0, nb = in ? n_b : 0;
      const uint8_t *ga = pa + (in ? iu * 128 : 0), *gb = pb + (in ? iu * 128 : 0);
      q.push(ga, gb, ga + up, gb + up, na, nb, na, nb);
      iu += 1 << ir.lg;
      if (__builtin_expect(iu >= KU, 0)) {
        next(ir);
        enter();
      }
    }
    q.commit();
  }
  __device__ __forceinline__ void start() {
    q.reset();
#pragma unroll 1
    for (int i = 1; i < q.depth; ++i) issue();
  }
  // h of feature i8 (0..7) of group gi for token t, from its gate and up sums
  __device__ __forceinline__ void finish(int gi, int i8, int t, float vg, float vu) const {
    const int u = u0 + 2 * gi + (i8 >> 2);
    if (u >= u1 || t >= a.T) return;
    const int ei = div_small(u, a.by_ui), f = (u - ei * UI) * 4 + (i8 & 3);
    const int sl = SHARED ? 0 : s.slot()[ei * 16 + t];
    if (sl < 0) return;
    const float h = vg / (1.0f + __expf(-vg)) * vu;
    const size_t row = SHARED ? size_t(t) : size_t(t) * a.k + sl;
    if (F8) {
      static_cast<float*>(a.h)[row * a.I + f] = h;
    } else {
      T16* o = static_cast<T16*>(SHARED ? a.h_sh : a.h) + row * 2 * a.I + f;
      const T16 hi = T16(h);
      o[0] = hi;
      o[a.I] = T16(isinf(float(hi)) ? 0.0f : h - float(hi));
    }
  }
  __device__ __forceinline__ void run() {
    const int KB = fp8_blocks(a.H);
    const uint8_t* xb[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = min(n * 8 + g, a.T - 1);  // columns past the last token repeat it; their results are not read
      xb[n] = s.x16() + size_t(t) * x16_pitch(a.H) + tig * 16;
    }
    Round r = {0, 0, 0};
    width_of(r);
#pragma unroll 1
    for (; r.first < groups; next(r)) {
      const int gi = group_of(r);
      float acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
      if (gi < groups && k0_of(r) < KU) {
        const float* psc = nullptr;
        int to_up = 0;
        if (F8) {
          psc = scales_of(min(u0 + 2 * gi + (g >> 2), u1 - 1));
          to_up = fp8_blocks(a.I) * KB;
        }
#pragma unroll 1
        for (int ku = k0_of(r); ku < KU; ku += 1 << r.lg) {
          const float2 sc = F8 ? make_float2(__ldg(psc + ku), __ldg(psc + to_up + ku)) : make_float2(1.0f, 1.0f);
          issue();
          const Unit w8 = q.pop();
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint8_t* xp = xb[n] + ku * 128 * (F8 ? 2 : 1);
            [[maybe_unused]] float d[4];
            if constexpr (F8) {
              // the second half of a partial unit is zero in the weights: x is read in place of what is not there
              const int off1 = ku * 128 + 64 >= row_bytes ? 0 : 128;
              const uint4 xv[4] = {*reinterpret_cast<const uint4*>(xp), *reinterpret_cast<const uint4*>(xp + 64),
                                   *reinterpret_cast<const uint4*>(xp + off1), *reinterpret_cast<const uint4*>(xp + off1 + 64)};
              unit_e4m3<KIND>(d, w8.lo0, w8.hi0, w8.lo1, w8.hi1, xv);
              const int c = n * 8 + 2 * tig;
              const float x0 = s.xsc()[min(c, a.T - 1) * KB + ku], x1 = s.xsc()[min(c + 1, a.T - 1) * KB + ku];
              acc[n][0] = fmaf(d[0], sc.x * x0, acc[n][0]);
              acc[n][1] = fmaf(d[1], sc.x * x1, acc[n][1]);
              acc[n][2] = fmaf(d[2], sc.y * x0, acc[n][2]);
              acc[n][3] = fmaf(d[3], sc.y * x1, acc[n][3]);
            } else {
              mma_half<KIND>(acc[n], w8.lo0, w8.hi0, *reinterpret_cast<const uint4*>(xp));
              mma_half<KIND>(acc[n], w8.lo1, w8.hi1, *reinterpret_cast<const uint4*>(xp + 64));
            }
          }
        }
      }
      if (r.lg == 0) {
        if (gi < groups) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            finish(gi, g, n * 8 + 2 * tig, acc[n][0], acc[n][2]);
            finish(gi, g, n * 8 + 2 * tig + 1, acc[n][1], acc[n][3]);
          }
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float* o = s.red() + (size_t(r.shared * kWarps + warp) * NT + n) * 128 + 2 * tig;
          *reinterpret_cast<float2*>(o + g * 8) = make_float2(acc[n][0], acc[n][1]);
          *reinterpret_cast<float2*>(o + (g + 8) * 8) = make_float2(acc[n][2], acc[n][3]);
        }
      }
    }
    // the shared rounds' groups: their warps' parts in warp order
    __syncthreads();
    r = {groups & ~(kWarps - 1), 0, 0};
    width_of(r);
#pragma unroll 1
    for (; r.first < groups; next(r)) {
      const int WG = 1 << r.lg, n = (kWarps >> r.lg) * 8 * a.T;
      int lgp = 0;
      while (lgp < r.lg && (n << (lgp + 1)) <= kThreads) ++lgp;
      const int P = 1 << lgp;
#pragma unroll 1
      for (int i0 = 0; i0 < n; i0 += kThreads >> lgp) {
        const int item = i0 + (threadIdx.x >> lgp), part = threadIdx.x & (P - 1);
        const int it = item < n ? item : 0;
        const int i8 = it & 7, gg = (it >> 3) & ((kWarps >> r.lg) - 1), t = (it >> 3) >> (4 - r.lg);
        const float* p = s.red() + (size_t(r.shared * kWarps + gg * WG) * NT + (t >> 3)) * 128 + i8 * 8 + (t & 7);
        float vg = 0.0f, vu = 0.0f;
        for (int w2 = part; w2 < WG; w2 += P) {
          vg += p[w2 * NT * 128];
          vu += p[w2 * NT * 128 + 64];
        }
        for (int o = P >> 1; o > 0; o >>= 1) {
          vg += __shfl_xor_sync(0xffffffffu, vg, o);
          vu += __shfl_xor_sync(0xffffffffu, vu, o);
        }
        if (item < n && part == 0 && r.first + gg < groups) finish(r.first + gg, i8, t, vg, vu);
      }
    }
    __syncthreads();
  }
};

// ---------------------------------------------------------------------------
// Output columns [n0, n0 + nrows), MT tiles of 16: the shared expert's K units,
// then the listed experts'.  Each warp takes an even run of consecutive units,
// so pointers advance by 128 bytes and an expert's products add up in place.
// The token operand holds only the tokens that selected the expert (one or two
// of sixteen, most often), and at the end of an expert's run f is weighted and
// added to the warp's sums of those tokens in shared memory.
// ---------------------------------------------------------------------------
template <typename T16, bool F8, int MT, int NT>
struct Down {
  static constexpr int KIND16 = MmaKind<T16>::v;
  const Args& a;
  const Smem& s;
  Queue& q;
  float* ysum;  // this warp's [T][16 MT]
  int n0, nrows, KS, KU, u0, u1, it0, ku0, g, tig;
  // issue position
  int iu, iit, iku, ilen, im;
  const uint8_t* ip;

  __device__ Down(const Args& a_, const Smem& s_, Queue& q_, float* ysum_, int nd, int n0_, int nrows_)
      : a(a_), s(s_), q(q_), ysum(ysum_), n0(n0_), nrows(nrows_) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    g = lane >> 2;
    tig = lane & 3;
    KS = a.sh_gu ? a.I / 64 : 0;
    KU = F8 ? fp8_blocks(a.I) : a.I / 64;
    const int units = nrows > 0 ? KS + nd * KU : 0;
    u0 = (units * warp) >> 4;
    u1 = (units * (warp + 1)) >> 4;
    it0 = u0 >= KS ? (F8 ? div_small(u0 - KS, a.by_ib) : div_small((u0 - KS) * 16, a.by_ui)) : -1;  // -1: shared
    ku0 = u0 >= KS ? u0 - KS - it0 * KU : u0;
    iu = u0;
    iit = it0;
    iku = ku0;
    im = 0;
    if (iu < u1) rows_of();
  }
  __device__ __forceinline__ void rows_of() {
    const bool sh = iit < 0;
    const int e = sh ? 0 : s.list()[iit];
    ilen = sh ? KS : KU;
    const int lane = threadIdx.x & 31;
    ip = (sh ? a.sh_d : a.w_d) + ((size_t(e) * a.H + n0 + (lane >> 3)) * a.I) * (sh || !F8 ? 2 : 1) + iku * 128 + (lane & 7) * 16;
  }
  __device__ __forceinline__ void issue() {
    if (iu < u1) {
      const bool wide = !F8 || iit < 0;
      const int pitch = a.I * (wide ? 2 : 1);
      const int lane = threadIdx.x & 31, left = nrows - im * 16 - (lane >> 3);  // rows left from this lane's first
      // 16-bit rows are whole 128-byte units (I is a multiple of 64)
      const bool in = wide || iku * 128 + (lane & 7) * 16 < a.I;
      const uint8_t* p = ip + im * 16 * pitch;
      // rows past the block's last are not copied: what the slot holds there reaches only results that nobody stores
      const uint32_t d = q.at(q.in) + q.wr, n = in ? 16 : 0;
      if (!in) p = ip;
      if (left > 0) cp_async_16(d, p, n);
      if (left > 4) cp_async_16(d + 512, p + 4 * pitch, n);
      if (left > 8) cp_async_16(d + 1024, p + 8 * pitch, n);
      if (left > 12) cp_async_16(d + 1536, p + 12 * pitch, n);
      if (++im == MT) {
        im = 0;
        ++iu;
        ip += 128;
        if (__builtin_expect(++iku == ilen, 0)) {
          iku = 0;
          ++iit;
          if (iu < u1) rows_of();
        }
      }
    }
    q.commit();
  }
  __device__ __forceinline__ void start() {
    q.reset();
#pragma unroll 1
    for (int i = 1; i < q.depth; ++i) issue();
  }
  // What an item's products need, for X columns of 8 tokens.  PACKED (16-bit,
  // at most 4 tokens): columns 0..3 take the high parts of h, 4..7 the low ones.
  template <int X>
  struct Item {
    int it, n;
    const uint8_t* hp[X];  // this lane's column, or null
    int sp[X];             // FP8: the token's scale row
    int wp[2 * MT];        // FP8: the weight rows' scales
  };
  template <bool WIDE, bool PACKED, int X>
  __device__ __forceinline__ void enter(Item<X>& e, int it, int n) const {
    const bool sh = it < 0;
    e.it = it;
    e.n = n;
    const uint8_t* hb = sh ? static_cast<const uint8_t*>(a.h_sh)
                           : (F8 ? (a.staged ? s.stage() : reinterpret_cast<const uint8_t*>(a.hq)) : static_cast<const uint8_t*>(a.h));
#pragma unroll
    for (int x = 0; x < X; ++x) {
      const int c = PACKED ? (g & 3) : x * 8 + g;
      e.hp[x] = nullptr;
      e.sp[x] = 0;
      if (c < n) {
        const int ent = sh ? 0 : s.ent()[it * 16 + c];
        const int row = sh ? c : (ent & 15) * a.k + (ent >> 4);
        e.hp[x] = hb + size_t(row) * a.I * (WIDE ? 4 : 2) + tig * 16 + (PACKED && g >= 4 ? 2 * a.I : 0);
        e.sp[x] = row * KU;
      }
    }
    if constexpr (!WIDE) {
#pragma unroll
      for (int m = 0; m < 2 * MT; ++m) {
        // rows past the block's last repeat it: their products are zero
        const int nb = (n0 + min(m * 8 + g, nrows - 1)) / kFp8Block;
        e.wp[m] = (s.list()[it] * fp8_blocks(a.H) + nb) * KU;
      }
    }
  }
  // One K unit of h: PACKED two halves; WIDE halves of the high, then of the low part; FP8 four pieces and the scales.
  template <bool WIDE, bool PACKED, int X>
  struct Frag {
    uint4 b[X][PACKED ? 2 : 4];
    float sc[WIDE ? 1 : X];
    float2 ws[WIDE ? 1 : MT];
  };
  template <bool WIDE, bool PACKED, int X>
  __device__ __forceinline__ void load(const Item<X>& e, int ku, Frag<WIDE, PACKED, X>& f) const {
    const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int x = 0; x < X; ++x) {
      const bool on = e.hp[x] != nullptr;
      const uint8_t* p = e.hp[x] + ku * (WIDE ? 128 : 256);
      f.b[x][0] = on ? *reinterpret_cast<const uint4*>(p) : z;
      f.b[x][1] = on ? *reinterpret_cast<const uint4*>(p + 64) : z;
      if constexpr (!PACKED) {
        const int off2 = WIDE ? 2 * a.I : 128;
        const bool on2 = on && (WIDE || ku * 128 + 64 < a.I);
        f.b[x][2] = on2 ? *reinterpret_cast<const uint4*>(p + off2) : z;
        f.b[x][3] = on2 ? *reinterpret_cast<const uint4*>(p + off2 + 64) : z;
      }
      if constexpr (!WIDE) {
        const float* hs = a.staged ? reinterpret_cast<const float*>(s.stage() + stage_scales(a.T, a.k, a.I)) : a.hs;
        f.sc[x] = on ? hs[e.sp[x] + ku] : 0.0f;
      }
    }
    if constexpr (!WIDE) {
#pragma unroll
      for (int m = 0; m < MT; ++m) f.ws[m] = make_float2(__ldg(a.sc_d + e.wp[2 * m] + ku), __ldg(a.sc_d + e.wp[2 * m + 1] + ku));
    }
  }
  template <bool WIDE, bool PACKED, int X>
  __device__ __forceinline__ void products(const Item<X>& e, const Frag<WIDE, PACKED, X>& f, float (&d)[MT][X][4]) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      issue();
      const Unit w = q.pop();
#pragma unroll
      for (int x = 0; x < X; ++x) {
        if (X > 1 && x * 8 >= e.n) continue;  // uniform in the warp
        float v[4];
        if constexpr (PACKED) {
          v[0] = v[1] = v[2] = v[3] = 0.0f;
          mma_half<KIND16>(d[m][x], w.lo0, w.hi0, f.b[x][0]);
          mma_half<KIND16>(v, w.lo1, w.hi1, f.b[x][1]);
#pragma unroll
          for (int j = 0; j < 4; ++j) d[m][x][j] += v[j];
        } else if constexpr (WIDE) {
          v[0] = v[1] = v[2] = v[3] = 0.0f;
          mma_half<KIND16>(d[m][x], w.lo0, w.hi0, f.b[x][0]);
          mma_half<KIND16>(v, w.lo0, w.hi0, f.b[x][2]);
          mma_half<KIND16>(d[m][x], w.lo1, w.hi1, f.b[x][1]);
          mma_half<KIND16>(v, w.lo1, w.hi1, f.b[x][3]);
#pragma unroll
          for (int j = 0; j < 4; ++j) d[m][x][j] += v[j];
        } else {
          unit_e4m3<MMA_F16>(v, w.lo0, w.hi0, w.lo1, w.hi1, f.b[x]);  // zeros past a partial unit
          const float h0 = __shfl_sync(0xffffffffu, f.sc[x], 8 * tig), h1 = __shfl_sync(0xffffffffu, f.sc[x], 8 * tig + 4);
          d[m][x][0] = fmaf(v[0], f.ws[m].x * h0, d[m][x][0]);
          d[m][x][1] = fmaf(v[1], f.ws[m].x * h1, d[m][x][1]);
          d[m][x][2] = fmaf(v[2], f.ws[m].y * h0, d[m][x][2]);
          d[m][x][3] = fmaf(v[3], f.ws[m].y * h1, d[m][x][3]);
        }
      }
    }
  }
  // Weights f and adds it to the warp's sums; d starts anew.
  template <bool PACKED, int X>
  __device__ __forceinline__ void leave(const Item<X>& e, float (&d)[MT][X][4]) {
    const bool sh = e.it < 0;
#pragma unroll
    for (int x = 0; x < X; ++x) {
      if (PACKED) {
        // column c + 4 (two lanes on) holds the low part of column c
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) d[m][x][j] += __shfl_xor_sync(0xffffffffu, d[m][x][j], 2);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = x * 8 + 2 * tig + i;
        if (c < e.n && !(PACKED && tig >= 2)) {
          const int ent = sh ? c : s.ent()[e.it * 16 + c];
          const int t = ent & 15;
          const float w = sh ? s.gate()[t] : s.sel_w()[t * kMaxSlots + (ent >> 4)];
          float* y = ysum + t * 16 * MT + g;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            y[m * 16] = fmaf(w, d[m][x][i], y[m * 16]);
            y[m * 16 + 8] = fmaf(w, d[m][x][2 + i], y[m * 16 + 8]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) d[m][x][0] = d[m][x][1] = d[m][x][2] = d[m][x][3] = 0.0f;
    }
  }
  __device__ __forceinline__ int tokens_of(int it) const { return it < 0 ? a.T : __popc(s.tmask()[it]); }
  // An item's units up to its end or the warp's.
  template <bool WIDE, bool PACKED, int X>
  __device__ __forceinline__ void run_item(int& u, int& it, int& ku) {
    Item<X> e;
    float d[MT][X][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int x = 0; x < X; ++x) d[m][x][0] = d[m][x][1] = d[m][x][2] = d[m][x][3] = 0.0f;
    enter<WIDE, PACKED, X>(e, it, tokens_of(it));
    const int end = min(u1 - u, (it < 0 ? KS : KU) - ku) + u;
    // h of the unit at hand only: asked for one unit ahead, it cost 0.4 us (16-bit, T = 1)
    // to 11 us (16 tokens) in registers and copies; the other warps cover its way from L2
#pragma unroll 1
    for (; u < end; ++u, ++ku) {
      Frag<WIDE, PACKED, X> f;
      load<WIDE, PACKED, X>(e, ku, f);
      products<WIDE, PACKED, X>(e, f, d);
    }
    leave<PACKED, X>(e, d);
    ku = 0;
    ++it;
  }
  __device__ __forceinline__ void run() {
    int u = u0, it = it0, ku = ku0;
#pragma unroll 1
    while (u < u1) {
      if constexpr (F8) {
        if (it < 0)
          run_item<true, false, NT>(u, it, ku);
        else
          run_item<false, false, NT>(u, it, ku);
      } else {
        // at most 4 tokens: the high and low parts of h side by side in one operand
        // (a T = 1 layer in 30.3 us against 31.5 through the wide form)
        if (tokens_of(it) <= 4)
          run_item<true, true, 1>(u, it, ku);
        else
          run_item<true, false, NT>(u, it, ku);
      }
    }
  }
};

// FP8: quantises (row, 128 features) blocks first, first + step, ... of h, one
// warp each, four at a time (their loads from L2 together).
__device__ void quant_h(const Args& a, __half* codes, float* scales, int first, int step) {
  const int IB = fp8_blocks(a.I), lane = threadIdx.x & 31, n = a.T * a.k * IB;
#pragma unroll 1
  for (int b0 = first; b0 < n; b0 += 4 * step) {
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = min(b0 + i * step, n - 1), row = div_small(b, a.by_ib), col = (b - row * IB) * kFp8Block + lane * 4;
      // columns past I repeat the row's first ones: they change no maximum
      v[i] = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(a.h) + size_t(row) * a.I +
                                                    (col < a.I ? col : (b - row * IB) * kFp8Block)));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = b0 + i * step, row = div_small(b, a.by_ib), col = (b - row * IB) * kFp8Block + lane * 4;
      float m = fmaxf(fmaxf(fabsf(v[i].x), fabsf(v[i].y)), fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const Fp8Scale sc = fp8_scale(m);
      if (b < n) {
        if (col < a.I)
          *reinterpret_cast<uint2*>(codes + size_t(row) * a.I + operand_order(col)) =
              e4m3x4_to_f16(fp8_quant4(v[i].x, v[i].y, v[i].z, v[i].w, sc.r));
        if (lane == 0) scales[b] = sc.s;
      }
    }
  }
}

// Columns [n0, n0 + nrows) of y, at most 16 MT; the rest of barrier 2 and the h
// rows' way into the operand form come between the requests and the products.
template <typename T16, bool F8, int MT, int NT>
__device__ __forceinline__ void columns(const Args& a, const Smem& s, cg::grid_group& grid,
                                        cg::grid_group::arrival_token&& token, int nd, int n0, int nrows) {
  const int warp = threadIdx.x >> 5;
  // nobody reads x any more: the warps' sums [16][T][16 MT] end where red ends, the queue takes what is before them
  uint8_t* const end = reinterpret_cast<uint8_t*>(s.red()) + kRedBytes;
  const int bytes = kWarps * a.T * 16 * MT * 4;
  float* ysum = reinterpret_cast<float*>(end - bytes);
  Queue q(s, a.depth, s.x16(), int(end - s.x16()) - max(bytes, kRedBytes));
  for (int i = threadIdx.x; i < bytes / 4; i += kThreads) ysum[i] = 0.0f;
  Down<T16, F8, MT, NT> down(a, s, q, ysum + warp * a.T * 16 * MT, nd, n0, nrows);
  down.start();
  grid.barrier_wait(std::move(token));
  if (F8) {
    __half* const codes = a.staged ? reinterpret_cast<__half*>(s.stage()) : a.hq;
    float* const scales = a.staged ? reinterpret_cast<float*>(s.stage() + stage_scales(a.T, a.k, a.I)) : a.hs;
    quant_h(a, codes, scales, a.staged ? warp : blockIdx.x + gridDim.x * warp, a.staged ? kWarps : gridDim.x * kWarps);
    if (!a.staged) grid.sync();
  }
  __syncthreads();  // the sums are zero, the codes written
  down.run();
  __syncthreads();
  // the warps' sums, in warp order
  const int n = 16 * MT * a.T, lgp = 31 - __clz(split_of(n)), P = 1 << lgp;
#pragma unroll 1
  for (int j0 = 0; j0 < n; j0 += kThreads >> lgp) {
    const int i = j0 + (threadIdx.x >> lgp), part = threadIdx.x & (P - 1);
    const int it = i < n ? i : 0;
    const int row = it & (16 * MT - 1), t = it / (16 * MT);
    float v = 0.0f;
    for (int w = part; w < kWarps; w += P) v += ysum[w * n + it];
    for (int o = P >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (i < n && part == 0 && row < nrows) static_cast<T16*>(a.y)[size_t(t) * a.H + n0 + row] = T16(v);
  }
  __syncthreads();
}

template <typename T16, bool F8, int NT, int MT>
__global__ void __launch_bounds__(kThreads, 1) k_layer_decode(const Args a) {
  cg::grid_group grid = cg::this_grid();
  const Smem s{a};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blk = blockIdx.x;
  const int T = a.T;
  Queue q(s, a.depth, s.queue(), 0);

  // ---- phase 0
  fetch_x(a, s);
  uint4 wr[kRouterPieces];
  router_fetch<T16>(a, blk, wr);
  const int2 su = a.sh_gu ? share_of(a.I / 4, a.by_grid) : make_int2(0, 0);
  GateUp<T16, false, NT, true> shared(a, s, a.sh_gu, q, su.x, su.y);
  shared.start();
  for (int i = tid; i < kMaxList * 4; i += kThreads) reinterpret_cast<uint32_t*>(s.slot())[i] = 0xffffffffu;
  if (tid < kMaxList) s.tmask()[tid] = 0;
  if (tid < 32) s.bits()[tid] = 0;
  cp_async_wait(q.depth - 1);  // x and the vectors: all but the shared expert's requests
  __syncthreads();
  if (a.norm_w) norm_x<T16>(a, s);
  shared_gate_value<T16>(a, s);
  if (a.gate_w) __syncthreads();  // the router's partial sums take the gate vector's place
  router<T16>(a, s, wr);
  auto token1 = grid.barrier_arrive();
  shared.run();
  if (F8) quant_x<T16>(a, s);
  grid.barrier_wait(std::move(token1));

  // ---- selection, by every block
  if (warp < T) {
    const float* row = a.logits + size_t(warp) * a.E;
    int* idx = s.sel_idx() + warp * kMaxSlots;
    float* w = s.sel_w() + warp * kMaxSlots;
    uint32_t* buf = reinterpret_cast<uint32_t*>(s.red()) + warp * 64;
    if (a.E <= 256) select_token<8>(row, a.E, a.k, lane, idx, w, buf);
    else if (a.E <= 512) select_token<16>(row, a.E, a.k, lane, idx, w, buf);
    else select_token<32>(row, a.E, a.k, lane, idx, w, buf);
  }
  __syncthreads();
  const int st = div_small(tid, a.by_k), sj = tid - st * a.k;
  int se = 0;
  if (tid < T * a.k) {
    se = s.sel_idx()[st * kMaxSlots + sj];
    atomicOr(s.bits() + (se >> 5), 1u << (se & 31));
  }
  __syncthreads();
  int nd;
  {
    // lane i counts word i; the experts below one's own are the words before it and its lower bits
    const uint32_t b = s.bits()[lane];
    int incl = __popc(b);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    nd = __shfl_sync(0xffffffffu, incl, 31);
    const int before = __shfl_sync(0xffffffffu, incl - __popc(b), se >> 5);
    if (tid < T * a.k) {
      const int below = before + __popc(s.bits()[se >> 5] & ((1u << (se & 31)) - 1u));
      s.list()[below] = se;
      s.slot()[below * 16 + st] = int8_t(sj);
      atomicOr(s.tmask() + below, 1u << st);
      if (blk == 0) {
        if (a.topk_idx) a.topk_idx[tid] = se;
        if (a.topk_w) a.topk_w[tid] = s.sel_w()[st * kMaxSlots + sj];
      }
      se = below;  // from here on: its place in the list
    }
  }
  __syncthreads();
  // read in phase 2, after the barriers on the way
  if (tid < T * a.k) s.ent()[se * 16 + __popc(s.tmask()[se] & ((1u << st) - 1u))] = uint8_t(st | (sj << 4));

  // ---- phase 1: gate/up
  {
    const int2 u = share_of(nd * (a.I / 4), a.by_grid);
    GateUp<T16, F8, NT, false> routed(a, s, a.w_gu, q, u.x, u.y);
    routed.start();
    routed.run();
  }
  auto token2 = grid.barrier_arrive();

  // ---- phase 2: down and the weighted sum
  const int2 col = share_of(a.H, a.by_grid);
  columns<T16, F8, MT, NT>(a, s, grid, std::move(token2), nd, col.x, col.y - col.x);
}

template <typename T16, bool F8, int NT, int MT>
int launch(Args a, cudaStream_t stream) {
  auto kern = k_layer_decode<T16, F8, NT, MT>;
  constexpr int kMaxDev = 64;
  static int blocks[kMaxDev] = {0};
  int dev = 0;
  MOE_CHECK_CUDA(cudaGetDevice(&dev));
  MOE_REQUIRE(dev < kMaxDev, MOE_ERR_UNSUPPORTED, "moe_layer_decode: device %d >= %d", dev, kMaxDev);
  if (blocks[dev] == 0) {
    // the largest size once: host threads may come here together
    MOE_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax));
    int per_sm = 0;
    MOE_CHECK_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, kSmemMax));
    MOE_REQUIRE(per_sm > 0, MOE_ERR_UNSUPPORTED, "moe_layer_decode: kernel does not fit on an SM");
    blocks[dev] = num_sms();
  }
  const size_t hb = F8 ? stage_bytes(a.T, a.k, a.I) : 0;
  auto room_of = [](size_t fixed) { return fixed < size_t(kSmemMax) ? (kSmemMax - fixed) / kSlotBytes : 0; };
  a.at = layout_of(a.T, a.H, F8, hb);
  a.staged = F8 && hb <= size_t(kStageBytes) && room_of(a.at.queue) >= 4;
  if (!a.staged) a.at = layout_of(a.T, a.H, F8, 0);
  const size_t fixed = a.at.queue;
  const size_t room = room_of(fixed);
  MOE_REQUIRE(room >= 2, MOE_ERR_UNSUPPORTED, "moe_layer_decode: T=%d H=%d do not fit in shared memory", a.T, a.H);
  a.depth = room > size_t(kMaxDepth) ? kMaxDepth : int(room);
  const size_t smem = fixed + size_t(a.depth) * kSlotBytes;
  a.by_ui = div_magic(a.I / 4);
  a.by_k = div_magic(a.k);
  a.by_grid = div_magic(blocks[dev]);
  a.by_ib = div_magic(fp8_blocks(a.I));
  void* params[] = {&a};
  MOE_CHECK_CUDA(cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kern), dim3(blocks[dev]), dim3(kThreads),
                                             params, smem, stream));
  return MOE_OK;
}

template <typename T16, bool F8, int NT>
int launch_mt(const Args& a, cudaStream_t stream) {
  // one 16-row tile where a block's columns fit in it: a second, empty one costs 2 to 10
  // us (BF16 T = 1 30.7 against 32.9, FP8 T = 8 63 against 74)
  return a.H <= 16 * num_sms() ? launch<T16, F8, NT, 1>(a, stream) : launch<T16, F8, NT, 2>(a, stream);
}
template <typename T16>
int dispatch(const Args& a, bool f8, cudaStream_t stream) {
  // FP8 up to 8 tokens: one 8-token operand in place of two (57 against 62 us at T = 8);
  // with 16-bit weights the second one costs nothing that could be measured
  if (f8) return a.T <= 8 ? launch_mt<T16, true, 1>(a, stream) : launch_mt<T16, true, 2>(a, stream);
  return launch_mt<T16, false, 2>(a, stream);
}

}  // namespace

// The sizes that the kernel takes: everything else is refused, and has no workspace size.
// A block holds at most two 16-row tiles of output columns, so H is also bounded by the SMs.
bool layer_decode_fits(int T, int H, int E, int k, int I) {
  return T >= 0 && T <= kLayerDecodeMaxT && H > 0 && H % 64 == 0 && H <= kLayerDecodeMaxH && T * H <= kLayerDecodeMaxTH &&
         I > 0 && I % 64 == 0 && I <= kLayerDecodeMaxI && k >= 1 && k <= kMaxSlots && k <= E && E <= kLayerDecodeMaxE &&
         H <= 32 * num_sms();
}

size_t layer_decode_ws_bytes(int T, int E, int k, int I) {
  WsCounter c;
  c.take<float>(size_t(T) * E);
  c.take<float>(size_t(T) * k * I);
  c.take<uint16_t>(size_t(T) * 2 * I);
  c.take<uint16_t>(size_t(T) * k * I);
  c.take<float>(size_t(T) * k * fp8_blocks(I));
  return c.used;
}

int layer_decode(const void* x, int T, int H, const void* norm_w, float eps, const void* w_shared_gate,
                 const void* w_router, const float* bias, int E, int k, int I, const void* w_gu, const float* sc_gu,
                 const void* w_d, const float* sc_d, bool f8, const void* w_sh_gu, const void* w_sh_d, int dtype,
                 int32_t* topk_idx, float* topk_w, void* y, void* ws, size_t ws_bytes, cudaStream_t stream) {
  Args a{};
  WsCarver carve(ws, ws_bytes);
  a.logits = carve.take<float>(size_t(T) * E);
  a.h = carve.take<float>(size_t(T) * k * I);
  a.h_sh = carve.take<uint16_t>(size_t(T) * 2 * I);
  a.hq = carve.take<__half>(size_t(T) * k * I);
  a.hs = carve.take<float>(size_t(T) * k * fp8_blocks(I));
  MOE_REQUIRE(carve.ok, MOE_ERR_WORKSPACE, "moe_layer_decode: workspace of %zu bytes is too small (need %zu)", ws_bytes,
              layer_decode_ws_bytes(T, E, k, I));
  a.x = x;
  a.T = T;
  a.H = H;
  a.E = E;
  a.k = k;
  a.I = I;
  a.norm_w = norm_w;
  a.eps = eps;
  a.gate_w = w_shared_gate;
  a.w_router = w_router;
  a.bias = bias;
  a.w_gu = static_cast<const uint8_t*>(w_gu);
  a.w_d = static_cast<const uint8_t*>(w_d);
  a.sc_gu = sc_gu;
  a.sc_d = sc_d;
  a.sh_gu = static_cast<const uint8_t*>(w_sh_gu);
  a.sh_d = static_cast<const uint8_t*>(w_sh_d);
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.y = y;
  return dtype == MOE_DTYPE_BF16 ? dispatch<__nv_bfloat16>(a, f8, stream) : dispatch<__half>(a, f8, stream);
}

}  // namespace moe
