// Persistent grouped GEMM on FP8 E4M3 operands with one FP32 scale per block
// of 128 along K (tcgen05.mma kind::f8f6f4, FP32 accumulate), and the expert
// FFN made of it.
//
//   out[r, n] = sum_kb sa[row(r), kb] * sw[g, n / 128, kb] * P_kb[r, n],
//   P_kb[r, n] = sum_{k in block kb} e4m3(A[row(r), k]) * e4m3(W[g, n, k])
//
// The scales are arbitrary FP32 numbers that change with every K block, so
// the tensor core's accumulator holds one block only: each K step of 128
// (one 128-byte swizzle row, four MMAs) starts a fresh accumulator in a ring
// of TMEM buffers, and eight promotion warps read it, multiply by the two
// scales and add into FP32 registers.  Per step of a 128 x 256 tile that is
// 128 FMAs for each of 256 threads against 4 MMAs of M = 128, N = 256, so the
// two run side by side.
//
// SwiGLU form: the tile holds 128 gate and the matching 128 up columns, which
// is one quantisation block of h per row: the epilogue forms h in FP32, takes
// the row's maximum (exchanged between the two warps that hold the row's
// halves) and writes E4M3 codes and the scale; h never goes to memory in 16
// bits.
//
// With row_token, A rows are gathered by four warps with cp.async straight
// into the 128-byte-swizzled A tile; rows past the group read zero.
//
// Warp roles: 0 TMA producer, 1 and 2 UMMA issuers of the even and the odd K
// steps (one thread's waits, issue and commits take about 800 cycles a step, the
// products 545; 1 owns the TMEM), 3 scales (row scale x column block scale of every
// step into shared memory, ahead of the promotion warps), 4..7 A-row gather, 8..15 promotion
// and epilogue (two per 32 rows, each half of the tile's columns).
//
// Measured: 8192 x 4096 x 2048 in 84 us in a burst (1650 TFLOP/s), 96 under load;
// 163840 rows x 2048 x 640 in 256 groups 353 and 425; the FFN of 8192 tokens, 512
// experts, k = 10, H = 2048, I = 640 602 and 729.  A K step takes 1320 cycles, its
// products 512, and no unit is busy half of the time (tensor pipe 38 %, packed FMAs
// 49 %, the products' operand reads 29 %): with two accumulators the order of a
// step's parts sets the pace.  Left out in copies of the dense product's 86.5 us:
// promotion and the output's way 57, the products too 45, the hand-overs too 40,
// which is the operands' way from L2 (48 KB a step in 590 cycles).
#include "fp8.cuh"
#include "gemm_sm100.cuh"

namespace moe {

int make_tmap_2d(CUtensorMap* map, const void* base, int rows, int cols, int esize, int box_rows, int box_cols,
                 CUtensorMapSwizzle swz);
int make_tmap_2d_u8_sw128(CUtensorMap* map, const void* base, int rows, int cols_bytes, int box_rows);
int fp8_quantize(const void* v, int batch, int rows, int K, int block_rows, int dtype, uint8_t* codes, float* scales,
                 cudaStream_t stream);

namespace {

constexpr int BM = 128;
constexpr int BK = kFp8Block;  // elements = bytes per row and K step
constexpr int A_BYTES = BM * BK;
constexpr int kThreads = 512;
constexpr int kGatherWarp0 = 4;
constexpr int kEpiWarp0 = 8;
constexpr int kSmemBudget = 212 * 1024;
// In place of the scale of a row without a token: a NaN that no product gives (those are
// 0x7fffffff), by which the epilogue finds the row.  The SwiGLU form takes 0 there, which
// makes the row zero for finite weights: the check would cost it registers (732 against
// 717 us on 8192 tokens), and its rows are promised no more.
constexpr uint32_t kNoRow = 0xffc0ffeeu;
constexpr int kStoreStride = 64 + 16;  // output staging: bytes per row of a 64-byte chunk, padded
constexpr int kBoxBytes = 32 * 128;    // 16-bit output: a box of 32 rows x 64 columns, two per warp
// registers per thread of the role groups: the sum over the four groups of
// 128 threads is what the block is launched with (512 x 128)
constexpr int kRegsIssue = 48, kRegsGather = 48, kRegsEpi = 208;
static_assert(kRegsIssue + kRegsGather + 2 * kRegsEpi == 4 * 128, "register split must equal the launch's total");

template <int BN, bool SWIGLU>
struct Cfg {
  static constexpr int B_BYTES = BN * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STORE_BYTES = SWIGLU ? 8 * 32 * kStoreStride : 8 * 2 * kBoxBytes;
  static constexpr int STAGES = (kSmemBudget - STORE_BYTES) / STAGE_BYTES;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + STORE_BYTES;
  static_assert(32 * kStoreStride <= 2 * kBoxBytes, "a warp's staging area serves both store forms");
  static constexpr int NACC = 512 / BN;  // TMEM accumulator ring
  static_assert(STAGE_BYTES % 1024 == 0, "stage must keep 1024-byte alignment");
};

struct Args {
  const int* group_offsets;  // [G+1] on the device, or null: one group of `rows` rows
  int G, rows, K, n_out, b_rows_per_group, up_offset;
  const float* sa;           // [a_rows, KB]
  const float* sw;           // [G, w_blocks, KB] (SwiGLU: [G, 2, w_blocks, KB])
  int w_blocks;
  void* out;                 // SwiGLU: E4M3 codes of h [rows, n_out]
  float* out_scales;         // SwiGLU: [rows, w_blocks]
  int out_kind;              // 0 BF16, 1 FP16, 2 FP32
  const int32_t* row_token;
  const uint8_t* a_src;      // [a_rows, K] codes
  int a_rows;
  int* status;
  unsigned long long limit_ns;
};

// kind::f8f6f4: D FP32, A and B E4M3 (0), K-major, M = 128
__host__ __device__ constexpr uint32_t idesc_e4m3(int N) {
  return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(BM >> 4) << 24);
}
__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_arrive_noinc(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// A TMEM load of 32 columns and its wait as two steps, so that the arithmetic on
// one chunk runs while the next is on its way.  The wait names the registers,
// which keeps their use behind it.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t ta, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%"
      "19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(ta)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// Two FP32 numbers in one register pair.
__device__ __forceinline__ uint64_t pack2(uint32_t a, uint32_t b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(a), "r"(b));
  return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ void fma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

// Stores a chunk of 64 bytes per row (one row per lane) through the warp's
// staging area: four lanes write one row's 64 bytes, eight rows an instruction,
// instead of 16 bytes of 32 rows.  Rows from nvalid on and bytes from nbytes on
// are left alone.
__device__ __forceinline__ void warp_store_64(uint8_t* stg, const uint32_t (&v)[16], int nvalid, int nbytes, uint8_t* gbase,
                                              size_t pitch, int lane) {
  uint4* mine = reinterpret_cast<uint4*>(stg + lane * kStoreStride);
#pragma unroll
  for (int i = 0; i < 4; ++i) mine[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  __syncwarp();
  const int seg = lane & 3;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int r = p * 8 + (lane >> 2);
    const uint4 w = *reinterpret_cast<const uint4*>(stg + r * kStoreStride + seg * 16);
    if (r < nvalid && seg * 16 < nbytes) st_global_v4(gbase + size_t(r) * pitch + seg * 16, w.x, w.y, w.z, w.w);
  }
  __syncwarp();
}

template <int R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// mbar_wait for the waits on the path from one K step to the next: polls
// instead of suspending.  Bounded the same way.
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                          unsigned long long limit_ns) {
  unsigned long long t0 = 0;
  for (uint32_t spins = 0;; ++spins) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((spins & 1023u) == 1023u) {
      const unsigned long long now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (*abort_flag) return false;
      if (now - t0 > limit_ns) {
        report(status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

struct TileMap {
  int g, m, n;
};

// Exclusive scan of the groups' row-tile counts into tile_start[0..G], row
// offsets into goff[0..G] (cut to the rows that exist).
__device__ void build_tile_table(const Args& a, int* goff, int* tile_start, int* warp_sums) {
  const int G = a.G, tid = threadIdx.x;
  for (int i = tid; i <= G; i += kThreads)
    goff[i] = a.group_offsets ? min(max(a.group_offsets[i], 0), a.rows) : (i == 0 ? 0 : a.rows);
  __syncthreads();
  const int per = (G + kThreads - 1) / kThreads;
  const int g0 = tid * per;
  int local = 0;
  for (int g = g0; g < g0 + per && g < G; ++g) {
    const int n = goff[g + 1] - goff[g];
    local += n > 0 ? (n + BM - 1) / BM : 0;
  }
  const int lane = tid & 31, warp = tid >> 5;
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int run = incl - local;
  for (int w = 0; w < warp; ++w) run += warp_sums[w];
  for (int g = g0; g < g0 + per && g < G; ++g) {
    tile_start[g] = run;
    const int n = goff[g + 1] - goff[g];
    run += n > 0 ? (n + BM - 1) / BM : 0;
  }
  if (tid == kThreads - 1) tile_start[G] = run;
  __syncthreads();
}

__device__ __forceinline__ TileMap decode_tile(int L, int nt, const int* tile_start, int G) {
  TileMap t;
  const int mt = L / nt;
  t.n = L - mt * nt;
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile_start[mid] <= mt) lo = mid; else hi = mid - 1;
  }
  t.g = lo;
  t.m = mt - tile_start[lo];
  return t;
}

template <int BN, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    k_grouped_gemm_fp8(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmO, const Args args) {
  using C = Cfg<BN, SWIGLU>;
  constexpr int STAGES = C::STAGES, NACC = C::NACC;
  constexpr int BNH = SWIGLU ? BN / 2 : BN;  // output columns per tile
  constexpr int NC = BN / 2;                 // accumulator columns per promotion thread
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[STAGES], empty_bar[STAGES], tfull_bar[NACC], tempty_bar[NACC], xbar[4],
      drain_bar[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ volatile int abort_flag;
  __shared__ int goff[kGemmMaxGroups + 1];
  __shared__ int tile_start[kGemmMaxGroups + 1];
  __shared__ int warp_sums[kThreads / 32];
  __shared__ float row_max[2][2][BM];
  __shared__ float step_scale[NACC][2][BM];  // of each accumulator: row scale x the two column blocks' scales

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto stg = [&](int s) { return smem + s * C::STAGE_BYTES; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool gathered = args.row_token != nullptr;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1 + (gathered ? 128 : 0));
      mbar_init(&empty_bar[s], 1);
    }
    for (int i = 0; i < NACC; ++i) {
      mbar_init(&tfull_bar[i], 2);   // the products' commit and the scale warp
      mbar_init(&tempty_bar[i], 8);  // one arrival per promotion warp
    }
    for (int i = 0; i < 4; ++i) mbar_init(&xbar[i], 2);  // the two warps of a row quadrant
    mbar_init(&drain_bar[0], 1);
    mbar_init(&drain_bar[1], 1);
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  // everything above touches no output of the kernel before
  griddep_wait();
  griddep_launch_dependents();
  build_tile_table(args, goff, tile_start, warp_sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_sh;

  const int G = args.G;
  const int nt = (args.n_out + BNH - 1) / BNH;
  const int total = tile_start[G] * nt;
  const int KB = fp8_blocks(args.K);
  int* status = args.status;
  const unsigned long long lim = args.limit_ns;

  if (warp < kGatherWarp0) {
    regs_dec<kRegsIssue>();
    if (warp == 0 && lane == 0) {
      // ---------------- TMA producer ----------------
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      bool ok = true;
      for (int L = blockIdx.x; L < total && ok; L += gridDim.x) {
        const TileMap t = decode_tile(L, nt, tile_start, G);
        const int a_row = goff[t.g] + t.m * BM;
        const int b_row = t.g * args.b_rows_per_group + t.n * BNH;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1, &abort_flag, status, lim)) { ok = false; break; }
          mbar_arrive_expect_tx(&full_bar[stage], (gathered ? 0 : A_BYTES) + C::B_BYTES);
          if (!gathered) tma_load_2d(stg(stage), &tmA, &full_bar[stage], kb * BK, a_row);
          tma_load_2d(stg(stage) + A_BYTES, &tmB, &full_bar[stage], kb * BK, b_row);
          if (SWIGLU)
            tma_load_2d(stg(stage) + A_BYTES + BNH * BK, &tmB, &full_bar[stage], kb * BK, b_row + args.up_offset);
          ++issued;
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) {
        volatile int never = 0;
        for (long i = (issued > STAGES ? issued - STAGES : 0); i < issued; ++i)
          mbar_wait(&full_bar[i % STAGES], uint32_t((i / STAGES) & 1), &never, nullptr, lim);
      }
    } else if ((warp == 1 || warp == 2) && lane == 0) {
      // ---------------- UMMA issuers ----------------
      // Steps are counted over all tiles; this thread issues those of its parity.
      constexpr uint32_t idesc = idesc_e4m3(BN);
      const long tiles = total > int(blockIdx.x) ? (total - int(blockIdx.x) + gridDim.x - 1) / gridDim.x : 0;
      const long steps = tiles * KB;
      for (long i = warp - 1; i < steps; i += 2) {
        const int stage = int(i % STAGES), buf = int(i % NACC);
        const uint32_t phase = uint32_t(i / STAGES) & 1, buf_phase = uint32_t(i / NACC) & 1;
        if (!mbar_poll(&tempty_bar[buf], buf_phase ^ 1, &abort_flag, status, lim) ||
            !mbar_poll(&full_bar[stage], phase, &abort_flag, status, lim))
          break;
        if (gathered) fence_proxy_async_smem();  // the gathered rows were written through the generic proxy
        tc_fence_after();
        const uint32_t sbase = smem_u32(stg(stage));
        const uint64_t ad = sdesc_kmajor_sw128(sbase), bd = sdesc_kmajor_sw128(sbase + A_BYTES);
        const uint32_t d = tmem_base + uint32_t(buf * BN);
#pragma unroll
        for (int j = 0; j < BK / 32; ++j)  // K = 32 per MMA: 32 bytes along the swizzled row
          umma_f8(d, ad + uint64_t(2 * j), bd + uint64_t(2 * j), idesc, j != 0);
        umma_commit(&tfull_bar[buf]);
        umma_commit(&empty_bar[stage]);
      }
      umma_commit(&drain_bar[warp - 1]);
      volatile int never = 0;
      mbar_wait(&drain_bar[warp - 1], 0, &never, nullptr, lim);
    }
    if (warp == 3) {
      // ---------------- scales ----------------
      int buf = 0;
      uint32_t buf_phase = 0;
      bool ok = true;
      for (int L = blockIdx.x; L < total && ok; L += gridDim.x) {
        const TileMap t = decode_tile(L, nt, tile_start, G);
        const int row0 = goff[t.g] + t.m * BM;
        const int tile_rows = min(BM, min(goff[t.g + 1], args.rows) - row0);
        int src[4];      // scale rows of tile rows lane, lane + 32, ..; -1: none
        float none[4];  // their scale: 0 past the tile's rows, which nobody stores
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane + 32 * i;
          int v = r < tile_rows ? row0 + r : -1;
          none[i] = !SWIGLU && v >= 0 ? __uint_as_float(kNoRow) : 0.0f;
          if (gathered && v >= 0) v = __ldg(args.row_token + v);
          src[i] = v >= 0 && v < args.a_rows ? v : -1;
        }
        // the two column blocks: gate and up, or the tile's halves
        const int nb0 = t.n * BNH / kFp8Block, nb1 = SWIGLU ? nb0 : min(nb0 + BN / 2 / kFp8Block, args.w_blocks - 1);
        const float* sw0 = args.sw + (size_t(t.g) * (SWIGLU ? 2 : 1) * args.w_blocks + nb0) * KB;
        const float* sw1 = args.sw + ((size_t(t.g) * (SWIGLU ? 2 : 1) + (SWIGLU ? 1 : 0)) * args.w_blocks + nb1) * KB;
        float a[4], w0 = __ldg(sw0), w1 = __ldg(sw1);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = src[i] >= 0 ? __ldg(args.sa + size_t(src[i]) * KB) : 0.0f;
        for (int kb = 0; kb < KB; ++kb) {
          float na[4] = {0.0f, 0.0f, 0.0f, 0.0f}, nw0 = 0.0f, nw1 = 0.0f;
          if (kb + 1 < KB) {
#pragma unroll
            for (int i = 0; i < 4; ++i) na[i] = src[i] >= 0 ? __ldg(args.sa + size_t(src[i]) * KB + kb + 1) : 0.0f;
            nw0 = __ldg(sw0 + kb + 1);
            nw1 = __ldg(sw1 + kb + 1);
          }
          if (!mbar_poll(&tempty_bar[buf], buf_phase ^ 1, &abort_flag, status, lim)) { ok = false; break; }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            step_scale[buf][0][lane + 32 * i] = src[i] >= 0 ? a[i] * w0 : none[i];
            step_scale[buf][1][lane + 32 * i] = src[i] >= 0 ? a[i] * w1 : none[i];
            a[i] = na[i];
          }
          w0 = nw0;
          w1 = nw1;
          __syncwarp();
          if (lane == 0) mbar_arrive(&tfull_bar[buf]);
          if (++buf == NACC) { buf = 0; buf_phase ^= 1; }
        }
      }
    }
  } else if (warp < kEpiWarp0) {
    regs_dec<kRegsGather>();
    if (gathered) {
      // ---------------- A row gather ----------------
      // Thread gt copies 16-byte chunk (gt % 8) of tile rows gt/8, gt/8 + 16, ...
      const int gt = threadIdx.x - kGatherWarp0 * 32;
      const int chunk = gt & 7, rbase = gt >> 3;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int L = blockIdx.x; L < total && ok; L += gridDim.x) {
        const TileMap t = decode_tile(L, nt, tile_start, G);
        const int a_row = goff[t.g] + t.m * BM;
        const int g_end = goff[t.g + 1];
        int tok[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = a_row + rbase + 16 * i;
          const int tk = (r < g_end && r < args.rows) ? __ldg(args.row_token + r) : -1;
          tok[i] = (tk >= 0 && tk < args.a_rows) ? tk : -1;
        }
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1, &abort_flag, status, lim)) { ok = false; break; }
          const uint32_t dst0 = smem_u32(stg(stage));
          const int k0 = kb * BK + chunk * 16;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = rbase + 16 * i;
            const uint32_t dst = dst0 + uint32_t(r * 128 + ((chunk ^ (r & 7)) << 4));
            const bool v = tok[i] >= 0 && k0 < args.K;
            cp_async_16_zfill(dst, args.a_src + (v ? size_t(tok[i]) * args.K + k0 : 0), v ? 16u : 0u);
          }
          cp_async_arrive_noinc(&full_bar[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // every copy has landed before the CTA exits
    }
  } else {
    regs_inc<kRegsEpi>();
    // ---------------- promotion and epilogue ----------------
    const int q = warp & 3;                   // TMEM lane quadrant: tile rows 32q .. 32q+31
    const int half = (warp - kEpiWarp0) >> 2; // column half
    const int row_in_tile = q * 32 + lane;
    int buf = 0;
    uint32_t buf_phase = 0, x_phase = 0;
    uint32_t box_no = 0;  // 16-bit output: this warp's boxes, over all tiles
    bool ok = true;
    for (int L = blockIdx.x; L < total && ok; L += gridDim.x) {
      const TileMap t = decode_tile(L, nt, tile_start, G);
      const int tile_rows = min(BM, min(goff[t.g + 1], args.rows) - (goff[t.g] + t.m * BM));
      const size_t out_row = size_t(goff[t.g]) + size_t(t.m) * BM + row_in_tile;
      const bool valid = row_in_tile < tile_rows;
      uint32_t row_scale = 0;
      // columns of this thread: output columns col0 .. (SwiGLU: BNH/2 of them, gate and up)
      const int col0 = t.n * BNH + half * (SWIGLU ? BNH / 2 : NC);
      const bool live = q * 32 < tile_rows && col0 < args.n_out;  // uniform in the warp
      const int nb = col0 / kFp8Block;
      uint64_t acc[NC / 2];  // pairs of neighbouring columns
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) acc[i] = 0;
      const uint32_t lane_base = tmem_base + (uint32_t(q * 32) << 16);
      for (int kb = 0; kb < KB; ++kb) {
        if (!mbar_poll(&tfull_bar[buf], buf_phase, &abort_flag, status, lim)) { ok = false; break; }
        tc_fence_after();
        if (live) {
          const uint32_t s0 = __float_as_uint(step_scale[buf][SWIGLU ? 0 : half][row_in_tile]);
          if (!SWIGLU) row_scale = s0;
          const uint32_t s1 = SWIGLU ? __float_as_uint(step_scale[buf][1][row_in_tile]) : s0;
          const uint64_t p0 = pack2(s0, s0), p1 = pack2(s1, s1);
          // SwiGLU: the first half of the chunks are gate columns, the rest the matching up columns
          constexpr int CH = NC / 32;
          auto col_of = [&](int c) {
            return SWIGLU ? (c < CH / 2 ? half * (BNH / 2) + 32 * c : BNH + half * (BNH / 2) + 32 * (c - CH / 2))
                          : half * NC + 32 * c;
          };
          const uint32_t tb = lane_base + uint32_t(buf * BN);
          // two chunks on their way at a time: the next two are requested as the registers come free
          uint32_t v[2][32];
          tmem_ld32_issue(tb + col_of(0), v[0]);
          tmem_ld32_issue(tb + col_of(1), v[1]);
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            if ((c & 1) == 0) {
              tmem_ld32_wait(v[0]);
              tmem_ld32_wait(v[1]);
              if (c + 2 == CH) {  // all columns are in registers: the buffer is free
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty_bar[buf]);
              }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              fma2(acc[16 * c + i], pack2(v[c & 1][2 * i], v[c & 1][2 * i + 1]), SWIGLU && c >= CH / 2 ? p1 : p0);
            if (c + 2 < CH) tmem_ld32_issue(tb + col_of(c + 2), v[c & 1]);
          }
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty_bar[buf]);
        }
        if (++buf == NACC) { buf = 0; buf_phase ^= 1; }
      }
      if (!ok) break;
      if (!SWIGLU && row_scale == kNoRow)  // zero, where a weight or its scale is not finite too
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) acc[i] = 0;
      uint8_t* stg_w = smem + STAGES * C::STAGE_BYTES + (warp - kEpiWarp0) * (SWIGLU ? 32 * kStoreStride : 2 * kBoxBytes);
      const int nvalid = tile_rows - q * 32;  // rows of this warp that exist
      const size_t row0 = size_t(goff[t.g]) + size_t(t.m) * BM + q * 32;
      if (SWIGLU) {
        constexpr int NH = NC / 2;  // h columns of this thread
        float h[NH];
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < NH / 2; ++i) {
          const float2 g = unpack2(acc[i]), u = unpack2(acc[NH / 2 + i]);
          h[2 * i] = __fdividef(g.x, 1.0f + __expf(-g.x)) * u.x;
          h[2 * i + 1] = __fdividef(g.y, 1.0f + __expf(-g.y)) * u.y;
          if (col0 + ((2 * i) & ~31) >= args.n_out) h[2 * i] = h[2 * i + 1] = 0.0f;  // n_out is a multiple of 64
          amax = fmaxf(amax, fmaxf(fabsf(h[2 * i]), fabsf(h[2 * i + 1])));
        }
        if (!live) amax = 0.0f;
        row_max[x_phase][half][row_in_tile] = amax;
        __syncwarp();
        if (lane == 0) mbar_arrive(&xbar[q]);
        if (!mbar_wait(&xbar[q], x_phase, &abort_flag, status, lim)) break;
        amax = fmaxf(amax, row_max[x_phase][half ^ 1][row_in_tile]);
        x_phase ^= 1;
        if (live) {
          const Fp8Scale s = fp8_scale(amax);
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) p[i] = fp8_quant4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3], s.r);
          warp_store_64(stg_w, p, nvalid, 64, static_cast<uint8_t*>(args.out) + row0 * args.n_out + col0, args.n_out, lane);
          if (half == 0 && valid) args.out_scales[out_row * args.w_blocks + nb] = s.s;
        }
      } else if (live) {
        if (args.out_kind == 2) {
#pragma unroll
          for (int c = 0; c < NC / 16; ++c) {
            if (col0 + 16 * c >= args.n_out) break;
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 f = unpack2(acc[8 * c + i]);
              p[2 * i] = __float_as_uint(f.x);
              p[2 * i + 1] = __float_as_uint(f.y);
            }
            warp_store_64(stg_w, p, nvalid, 64, static_cast<uint8_t*>(args.out) + (row0 * args.n_out + col0 + 16 * c) * 4,
                          size_t(args.n_out) * 4, lane);
          }
        } else {
          // boxes of 32 rows x 64 columns: written to shared memory in the 128-byte
          // swizzle and copied out by the tensor copy unit (whole lines, and the warp
          // goes on), or by the warp where rows are missing (they belong to the next
          // group).  A warp's two boxes take turns over all its tiles, not within one: a
          // half of a tile may hold a single box (BN = 128, or the last columns), and the
          // one copy that may still be reading has to be the other box's.
          auto store16 = [&](auto pack) {
#pragma unroll
            for (int c = 0; c < NC / 64; ++c) {
              if (col0 + 64 * c >= args.n_out) break;
              uint8_t* box = stg_w + (box_no & 1) * kBoxBytes;
              ++box_no;
              if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the copy before last has read
              __syncwarp();
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                uint32_t p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = pack(unpack2(acc[32 * c + 4 * k + i]));
                *reinterpret_cast<uint4*>(box + lane * 128 + ((k ^ (lane & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
              }
              if (nvalid >= 32) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                                   reinterpret_cast<uint64_t>(&tmO)),
                               "r"(smem_u32(box)), "r"(col0 + 64 * c), "r"(int(row0))
                               : "memory");
              } else {
                __syncwarp();
                const int seg = lane & 7;
                uint8_t* dst = static_cast<uint8_t*>(args.out) + (row0 * args.n_out + col0 + 64 * c) * 2 + seg * 16;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const int r = k * 4 + (lane >> 3);
                  const uint4 w = *reinterpret_cast<const uint4*>(box + r * 128 + ((seg ^ (r & 7)) << 4));
                  if (r < nvalid && col0 + 64 * c + seg * 8 < args.n_out)
                    st_global_v4(dst + size_t(r) * args.n_out * 2, w.x, w.y, w.z, w.w);
                }
              }
              if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          };
          if (args.out_kind == 0)
            store16([](float2 f) { return Pack2<__nv_bfloat16>::pack(f.x, f.y); });
          else
            store16([](float2 f) { return Pack2<__half>::pack(f.x, f.y); });
        }
      }
    }
  }

  if (!SWIGLU && warp >= kEpiWarp0 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <int BN, bool SWIGLU>
int launch(const Args& a, const uint8_t* w, int w_rows, cudaStream_t stream) {
  CUtensorMap ta, tb;
  int rc = make_tmap_2d_u8_sw128(&ta, a.a_src, a.a_rows, a.K, BM);
  if (rc) return rc;
  rc = make_tmap_2d_u8_sw128(&tb, w, w_rows, a.K, SWIGLU ? BN / 2 : BN);
  if (rc) return rc;
  CUtensorMap to = ta;  // only 16-bit outputs are stored through a map
  if (!SWIGLU && a.out_kind != 2) {
    rc = make_tmap_2d(&to, a.out, a.rows, a.n_out, 2, 32, 64, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
  }
  auto kern = k_grouped_gemm_fp8<BN, SWIGLU>;
  static bool attr_set[64] = {false};
  int dev = 0;
  MOE_CHECK_CUDA(cudaGetDevice(&dev));
  if (dev >= 64 || !attr_set[dev]) {
    MOE_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BN, SWIGLU>::SMEM_BYTES));
    if (dev < 64) attr_set[dev] = true;
  }
  MOE_CHECK_CUDA(launch_pdl(kern, dim3(num_sms()), dim3(kThreads), Cfg<BN, SWIGLU>::SMEM_BYTES, stream, ta, tb, to, a));
  return MOE_OK;
}

}  // namespace

// out [rows, N] = the grouped product of a [a_rows, K] and w [E, N, K].
int grouped_gemm_fp8(const uint8_t* a, const float* a_scales, int a_rows, const int32_t* row_token,
                     const int32_t* offsets, int rows, int K, int N, int E, const uint8_t* w, const float* w_scales,
                     int out_kind, void* out, cudaStream_t stream) {
  Args g{};
  g.group_offsets = offsets;
  g.G = E;
  g.rows = rows;
  g.K = K;
  g.n_out = N;
  g.b_rows_per_group = N;
  g.sa = a_scales;
  g.sw = w_scales;
  g.w_blocks = fp8_blocks(N);
  g.out = out;
  g.out_kind = out_kind;
  g.row_token = row_token;
  g.a_src = a;
  g.a_rows = a_rows;
  g.status = device_status_ptr();
  g.limit_ns = wait_limit_ns();
  // the wide tile where an upper bound of its tiles still covers the SMs: it reads the
  // A operand half as often (8192 x 4096 x 2048 in 83 us against 96, 163840 rows of 256
  // groups 353 against 436); fewer tiles than SMs leave some of them idle (640 rows of
  // 512 groups: 105 against 106 us, even)
  const long mt = (rows + BM - 1) / BM + (E < rows ? E : rows);
  if (mt * ((N + 255) / 256) >= num_sms()) return launch<256, false>(g, w, E * N, stream);
  return launch<128, false>(g, w, E * N, stream);
}

size_t fp8_swiglu_ws_bytes(int T, int rows, int H, int I) {
  WsCounter c;
  c.take<uint8_t>(size_t(T) * H);
  c.take<float>(size_t(T) * fp8_blocks(H));
  c.take<uint8_t>(size_t(rows) * I);
  c.take<float>(size_t(rows) * fp8_blocks(I));
  return c.used;
}

int grouped_swiglu_fp8(const void* x, const int32_t* row_token, const int32_t* offsets, int T, int rows, int H, int I,
                       int E, const uint8_t* w_gu, const float* sc_gu, const uint8_t* w_d, const float* sc_d,
                       int dtype, int out_fp32, void* f, void* ws, size_t ws_bytes, cudaStream_t stream) {
  WsCarver carve(ws, ws_bytes);
  uint8_t* xq = carve.take<uint8_t>(size_t(T) * H);
  float* xs = carve.take<float>(size_t(T) * fp8_blocks(H));
  uint8_t* hq = carve.take<uint8_t>(size_t(rows) * I);
  float* hs = carve.take<float>(size_t(rows) * fp8_blocks(I));
  MOE_REQUIRE(carve.ok, MOE_ERR_WORKSPACE, "moe_grouped_swiglu_fp8_b128: workspace of %zu bytes is too small (need %zu)",
              ws_bytes, fp8_swiglu_ws_bytes(T, rows, H, I));
  int rc = fp8_quantize(x, 1, T, H, 1, dtype, xq, xs, stream);
  if (rc) return rc;
  Args g{};
  g.group_offsets = offsets;
  g.G = E;
  g.rows = rows;
  g.K = H;
  g.n_out = I;
  g.b_rows_per_group = 2 * I;
  g.up_offset = I;
  g.sa = xs;
  g.sw = sc_gu;
  g.w_blocks = fp8_blocks(I);
  g.out = hq;
  g.out_scales = hs;
  g.row_token = row_token;
  g.a_src = xq;
  g.a_rows = T;
  g.status = device_status_ptr();
  g.limit_ns = wait_limit_ns();
  rc = launch<256, true>(g, w_gu, E * 2 * I, stream);
  if (rc) return rc;
  return grouped_gemm_fp8(hq, hs, rows, nullptr, offsets, rows, I, H, E, w_d, sc_d,
                          out_fp32 ? 2 : (dtype == MOE_DTYPE_BF16 ? 0 : 1), f, stream);
}

}  // namespace moe
