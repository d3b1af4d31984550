// Y = X W^T of two microscaled 4-bit matrices (include/gptq_mx.h) on the fifth-generation
// tensor cores: tcgen05.mma kind::mxf4 multiplies the codes and applies both sides' scales
// (one per 32 columns) itself, so nothing is dequantised.
//
// The MMA's M side is W (128 rows of the layer per tile) and its N side the tokens, so that
// one token costs an N = 16 tile and a thread of the epilogue holds one layer row, whose
// neighbours in a warp are neighbours in Y's rows.  K runs in stages of 256 columns: 128
// bytes of codes per row (TMA, 128-byte swizzle) and two 512-byte scale tiles per 128 rows.
// The scales reach TMEM with tcgen05.cp; every stage of the ring has TMEM columns of its own
// for them, so they are overwritten only after the MMAs that read them have released the
// stage.  Per CTA: warp 0 producer, warp 1 TMEM and MMA, warps 2-5 epilogue.
// Every mbarrier wait is bounded; a wait that gives up sets GPTQ_ERR_TIMEOUT and the CTA
// drains its own copies and MMAs before it frees TMEM and exits.
#include <algorithm>

#include "kernels.h"
#include "mx.cuh"
#include "tc_common.cuh"

namespace gptq {
namespace {

constexpr int TM = 128;                 // layer rows per tile
constexpr int KB = 128;                 // bytes of codes per row and stage: 256 columns
constexpr int A_BYTES = TM * KB;
constexpr int THREADS = 192;

template <int BN>
struct Cfg {
  static constexpr int NB = (BN + 127) / 128;                 // scale tiles of the token side
  static constexpr int B_BYTES = BN * KB;
  static constexpr int S_BYTES = (1 + NB) * 1024;             // both scale tiles of each 128 rows
  static constexpr int STAGE = A_BYTES + B_BYTES + S_BYTES;   // a multiple of 1024
  static constexpr int STAGES = 200 * 1024 / STAGE < 6 ? 200 * 1024 / STAGE : 6;
  static constexpr int SF_COLS = 8 * (1 + NB);                // TMEM columns of a stage's scales
  static constexpr int COLS = BN + STAGES * SF_COLS;
  static constexpr uint32_t TMEM_COLS = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static constexpr int SMEM = STAGES * STAGE + 1024 + 256;
  static_assert(COLS <= 512, "TMEM");
};

struct Prob {
  const uint8_t* xs;
  const uint8_t* ws;
  void* Y;
  int64_t ldy;
  int M, R;          // tokens, layer rows
  int steps;         // MMAs along K: 64 columns each
  int ct;            // scale tiles along K
  uint32_t wait_limit;
};

template <int BN, typename T>
__global__ void __launch_bounds__(THREADS, 1)
k_mx_matmul(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
            Prob p, uint32_t idesc, int32_t* status) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = blockIdx.x * TM, n0 = blockIdx.y * BN;
  const int nk = (p.steps + 3) >> 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(empty + i, 1);
    }
    tc::mbar_init(acc_full, 1);
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, C::TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  int64_t issued = 0;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      // scale tiles of the token side that exist: a 256-token tile may hold one only
      const int nbt = min(C::NB, (p.M + 127) / 128 - n0 / 128);
      for (int k = 0; k < nk; ++k) {
        if (!tc::mbar_wait(empty + stage, phase ^ 1u, abort_flag, p.wait_limit)) break;
        uint8_t* a = smem + stage * C::STAGE;
        uint8_t* s = a + A_BYTES + C::B_BYTES;
        const uint32_t sb = uint32_t(min(2, p.ct - 2 * k)) * 512;
        tc::mbar_expect_tx(full + stage, uint32_t(A_BYTES + C::B_BYTES) + sb * (1 + nbt));
        tc::tma_load_2d(a, &wmap, k * KB, r0, full + stage);
        tc::tma_load_2d(a + A_BYTES, &xmap, k * KB, n0, full + stage);
        tc::bulk_load(s, p.ws + (int64_t(blockIdx.x) * p.ct + 2 * k) * 512, sb, full + stage);
        for (int j = 0; j < nbt; ++j)
          tc::bulk_load(s + 1024 * (1 + j),
                        p.xs + (int64_t(n0 / 128 + j) * p.ct + 2 * k) * 512, sb, full + stage);
        ++issued;
        if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int k = 0; k < nk; ++k) {
        if (!tc::mbar_wait(full + stage, phase, abort_flag, p.wait_limit)) { ok = false; break; }
        tc::fence_after_sync();
        const uint8_t* a = smem + stage * C::STAGE;
        const uint8_t* b = a + A_BYTES;
        const uint8_t* s = b + C::B_BYTES;
        const uint32_t sfa = tmem_base + uint32_t(BN + stage * C::SF_COLS);
        const uint32_t sfb = sfa + 8;
        const int tiles = min(2, p.ct - 2 * k);
        for (int t = 0; t < tiles; ++t) {
          tc::copy_scales(sfa + 4 * t, tc::smem_desc_rows16(s + 512 * t));
#pragma unroll
          for (int j = 0; j < C::NB; ++j)
            tc::copy_scales(sfb + 4 * C::NB * t + 4 * j,
                            tc::smem_desc_rows16(s + 1024 * (1 + j) + 512 * t));
        }
        const int todo = min(4, p.steps - 4 * k);
        // a token tile of 32 or 64 starts inside its scale tile, 32 rows to a TMEM column
        const uint32_t sfb0 = sfb + uint32_t((n0 & 127) >> 5);
        for (int kk = 0; kk < todo; ++kk)
          tc::mma_mxf4(tmem_base, tc::smem_desc_sw128(a + kk * 32, 16, 1024),
                       tc::smem_desc_sw128(b + kk * 32, 16, 1024),
                       idesc | ((kk & 1) ? (2u << 4) | (2u << 29) : 0u), sfa + 4 * (kk >> 1),
                       sfb0 + 4 * C::NB * (kk >> 1), (k > 0 || kk > 0) ? 1u : 0u);
        tc::mma_commit(empty + stage);
        if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
      }
      if (ok) tc::mma_commit(acc_full);
    }
  } else {
    const int lane_base = (warp & 3) * 32;
    const int row = r0 + lane_base + lane;
    if (tc::mbar_wait(acc_full, 0, abort_flag, p.wait_limit)) {
      tc::fence_after_sync();
      for (int c = 0; c < BN; c += 16) {
        uint32_t v[16];
        tc::tmem_ld_32x16(tmem_base + (uint32_t(lane_base) << 16) + uint32_t(c), v);
        tc::tmem_ld_wait();
        T* y = static_cast<T*>(p.Y) + int64_t(n0 + c) * p.ldy + row;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (row < p.R && n0 + c + i < p.M) y[i * p.ldy] = from_f32<T>(__uint_as_float(v[i]));
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (*abort_flag) {
    if (warp == 0 && lane == 0) tc::drain_tma_ring(full, C::STAGES, issued);
    if (warp == 1 && lane == 0) {
      tc::mma_commit(drain);
      tc::mbar_drain(drain, 0);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0) raise_status(status, GPTQ_ERR_TIMEOUT);
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

bool encode_codes(CUtensorMap* m, const uint32_t* codes, uint64_t row_bytes, uint64_t rows,
                  uint32_t box_rows) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {row_bytes, rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {uint32_t(KB), box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint32_t*>(codes), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, typename T>
gptq_status launch(cudaStream_t st, const uint32_t* xc, const uint32_t* wc, uint64_t row_bytes,
                   const Prob& p, int32_t* status) {
  using C = Cfg<BN>;
  CUtensorMap wmap, xmap;
  if (!encode_codes(&wmap, wc, row_bytes, uint64_t(p.R), TM) ||
      !encode_codes(&xmap, xc, row_bytes, uint64_t(p.M), BN))
    return GPTQ_ERR_UNSUPPORTED;
  // idesc: 4-bit codes on both sides, K-major, byte scales 2^(e-127), N = BN, M = 128
  const uint32_t idesc = (1u << 7) | (1u << 10) | (uint32_t(BN >> 3) << 17) | (1u << 23) |
                         (uint32_t(TM >> 4) << 24);
  GPTQ_CUDA(allow_smem(k_mx_matmul<BN, T>, C::SMEM));
  const dim3 grid((p.R + TM - 1) / TM, (p.M + BN - 1) / BN);
  GPTQ_LAUNCH((k_mx_matmul<BN, T>), grid, THREADS, C::SMEM, st, wmap, xmap, p, idesc, status);
  return GPTQ_OK;
}

template <typename T>
gptq_status by_tokens(cudaStream_t st, const uint32_t* xc, const uint32_t* wc, uint64_t row_bytes,
                      const Prob& p, int32_t* status) {
  if (p.M <= 16) return launch<16, T>(st, xc, wc, row_bytes, p, status);
  if (p.M <= 32) return launch<32, T>(st, xc, wc, row_bytes, p, status);
  if (p.M <= 64) return launch<64, T>(st, xc, wc, row_bytes, p, status);
  if (p.M <= 128) return launch<128, T>(st, xc, wc, row_bytes, p, status);
  return launch<256, T>(st, xc, wc, row_bytes, p, status);
}

}  // namespace

gptq_status mx_matmul_run(cudaStream_t st, const uint32_t* xc, const uint8_t* xs, int M,
                          const uint32_t* wc, const uint8_t* ws, int R, int C, void* Y, int dt,
                          int64_t ldy, int32_t* status) {
  const int nb = (C + 31) / 32;
  Prob p;
  p.xs = xs;
  p.ws = ws;
  p.Y = Y;
  p.ldy = ldy;
  p.M = M;
  p.R = R;
  p.steps = (nb + 1) / 2;
  p.ct = (nb + 3) / 4;
  p.wait_limit = pipeline_wait_limit();
  const uint64_t row_bytes = uint64_t(nb) * 16;
  switch (dt) {
    case GPTQ_F32: return by_tokens<float>(st, xc, wc, row_bytes, p, status);
    case GPTQ_F16: return by_tokens<__half>(st, xc, wc, row_bytes, p, status);
    default: return by_tokens<__nv_bfloat16>(st, xc, wc, row_bytes, p, status);
  }
}

}  // namespace gptq
