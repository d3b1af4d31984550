// Y = X W^T of two microscaled 4-bit matrices (include/gptq_mx.h) on the fifth-generation
// tensor cores: tcgen05.mma kind::mxf4 multiplies the codes and applies both sides' scales
// (one per 32 columns) itself, so nothing is dequantised.
//
// The MMA's M side is W and its N side the tokens, so that few tokens cost a narrow tile and
// a thread of the epilogue holds one layer row, whose neighbours in a warp are neighbours in
// Y's rows.  K runs in boxes of 256 columns: 128 bytes of codes per row (TMA, 128-byte
// swizzle) and two 512-byte scale tiles per 128 rows.  The scales reach TMEM with tcgen05.cp;
// every stage of the ring has TMEM columns of its own for them, so they are overwritten only
// after the MMAs that read them have released the stage.
//
// Two kernels:
//  k_mx_few    128 layer rows x up to 64 tokens per CTA, K split over the CTAs of a cluster,
//              whose partial sums meet in distributed shared memory in a fixed order: few
//              tokens, where the weights' bytes are the work and row tiles alone would leave
//              SMs idle.
//  k_mx_pair   256 layer rows x up to 256 tokens per CTA pair (cta_group::2), persistent:
//              many tokens; where the tiles are few, up to four pairs share a tile's K in the
//              same way.
// Every mbarrier wait is bounded; a wait that gives up sets GPTQ_ERR_TIMEOUT and the CTA
// drains its own copies and MMAs before it frees TMEM and exits.
#include <algorithm>

#include "acc_ring.h"
#include "kernels.h"
#include "mx.cuh"
#include "tc_common.cuh"

namespace gptq {
namespace {

constexpr int KB = 128;                 // bytes of codes per row and box: 256 columns
constexpr int A_BOX = 128 * KB;

struct Prob {
  const uint8_t* xs;
  const uint8_t* ws;
  void* Y;
  int64_t ldy;
  int M, R;          // tokens, layer rows
  int steps;         // MMAs along K: 64 columns each
  int ct;            // scale tiles along K: 128 columns each
  int boxes;         // boxes along K: 256 columns each
  uint32_t wait_limit;
  int give_up;       // stage of a tile at which the last MMA issuer gives up (-1: none)
  // k_mx_pair only
  int bn;            // tokens of a tile, a multiple of 64
  int nb;            // scale tiles that a token tile touches
  int accs;          // accumulators
  int stages;        // of the ring
  int ntr, ntt;      // tiles along the layer rows and the tokens
};

// sf_id of both operands for the odd 64-column half of a scale tile: bytes 2 and 3
constexpr uint32_t ODD_HALF = (2u << 4) | (2u << 29);

// idesc: 4-bit codes on both sides, K-major, byte scales 2^(e-127)
constexpr uint32_t idesc_of(int m, int n) {
  return (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (1u << 23) | (uint32_t(m >> 4) << 24);
}

// ------------------------------------------------------------------ few tokens
constexpr int FEW_THREADS = 192;        // warp 0 producer, warp 1 TMEM and MMA, 2-5 epilogue

template <int BN>
struct Few {
  static constexpr int SUB = 2;                               // boxes of a stage
  static constexpr int B_BOX = BN * KB;
  static constexpr int S_BOX = 1024;                          // scales of 128 rows and a box
  static constexpr int STAGE = SUB * (A_BOX + B_BOX + 2 * S_BOX);
  static constexpr int STAGES = 200 * 1024 / STAGE < 6 ? 200 * 1024 / STAGE : 6;
  static constexpr int SF_COLS = SUB * 16;                    // TMEM columns of a stage's scales
  static constexpr int COLS = BN + STAGES * SF_COLS;
  static constexpr uint32_t TMEM_COLS = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static constexpr int SMEM = STAGES * STAGE + 1024 + 256;
  static_assert(COLS <= 512 && BN * 512 <= STAGES * STAGE, "TMEM, partial sums");
};

// BN: the token tile, all of the M <= BN tokens
template <int BN, typename T>
__global__ void __launch_bounds__(FEW_THREADS, 1)
k_mx_few(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
         Prob p, int32_t* status) {
  using C = Few<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::STAGES * C::STAGE);
  uint64_t* empty = full + C::STAGES;
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int split = int(tc::cluster_rank()), splits = int(tc::cluster_size());
  const int rt = blockIdx.x / splits;
  const int r0 = rt * 128;
  const int b0 = int(int64_t(p.boxes) * split / splits);
  const int b1 = int(int64_t(p.boxes) * (split + 1) / splits);

  if (threadIdx.x == 32) {
    tc::prefetch_map(&wmap);
    tc::prefetch_map(&xmap);
  }
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

  allow_successor();
  wait_for_predecessor();
  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    for (int b = b0; b < b1; b += C::SUB) {
      if (!tc::mbar_wait_warp(empty + stage, phase ^ 1u, abort_flag, p.wait_limit)) break;
      const int nbx = min(C::SUB, b1 - b);
      uint8_t* a = smem + stage * C::STAGE;
      uint8_t* x = a + C::SUB * A_BOX;
      uint8_t* s = x + C::SUB * C::B_BOX;
      const uint32_t sb = uint32_t(min(2 * nbx, p.ct - 2 * b)) * 512;
      if (tc::elect_one()) {
        tc::mbar_expect_tx(full + stage, uint32_t(nbx * (A_BOX + C::B_BOX)) + 2 * sb);
        for (int j = 0; j < nbx; ++j)
          tc::tma_load_2d(a + j * A_BOX, &wmap, (b + j) * KB, r0, full + stage);
        tc::bulk_load(s, p.ws + (int64_t(rt) * p.ct + 2 * b) * 512, sb, full + stage);
        for (int j = 0; j < nbx; ++j)
          tc::tma_load_2d(x + j * C::B_BOX, &xmap, (b + j) * KB, 0, full + stage);
        tc::bulk_load(s + C::SUB * C::S_BOX, p.xs + int64_t(2 * b) * 512, sb, full + stage);
      }
      __syncwarp();
      ++issued;
      if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
    }
  } else if (warp == 1) {
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    constexpr uint32_t idesc = idesc_of(128, BN);
    const int last = p.give_up >= 0 && split == splits - 1 ? b0 + C::SUB * p.give_up : b1;
    const uint64_t adesc0 = tc::smem_desc_sw128(smem, 16, 1024);
    const uint64_t sdesc0 = tc::smem_desc_rows16(smem + C::SUB * (A_BOX + C::B_BOX));
    for (int b = b0; b < b1; b += C::SUB) {
      ok = tc::mbar_wait_warp(full + stage, phase, abort_flag, b < last ? p.wait_limit : 0u);
      if (!ok) break;
      tc::fence_after_sync();
      // descriptors count in 16 bytes
      const uint64_t ad = adesc0 + uint32_t(stage) * (C::STAGE >> 4);
      const uint64_t xd = ad + (C::SUB * A_BOX >> 4);
      const uint64_t sd = sdesc0 + uint32_t(stage) * (C::STAGE >> 4);
      const uint32_t sfa = tmem_base + uint32_t(BN + stage * C::SF_COLS);
      const uint32_t sfb = sfa + 8 * C::SUB;
      const int tiles = min(2 * C::SUB, min(2 * (b1 - b), p.ct - 2 * b));
      const int todo = min(4 * C::SUB, min(4 * (b1 - b), p.steps - 4 * b));
      if (tc::elect_one()) {
#pragma unroll
        for (int t = 0; t < 2 * C::SUB; ++t)
          if (t < tiles) {
            tc::copy_scales(sfa + 4 * t, sd + 32 * t);
            tc::copy_scales(sfb + 4 * t, sd + (C::SUB * C::S_BOX >> 4) + 32 * t);
          }
#pragma unroll
        for (int kk = 0; kk < 4 * C::SUB; ++kk)
          if (kk < todo)
            tc::mma_mxf4(tmem_base, ad + (kk >> 2) * (A_BOX >> 4) + (kk & 3) * 2,
                         xd + (kk >> 2) * (C::B_BOX >> 4) + (kk & 3) * 2,
                         idesc | ((kk & 1) ? ODD_HALF : 0u), sfa + 4 * (kk >> 1),
                         sfb + 4 * (kk >> 1), (b > b0 || kk > 0) ? 1u : 0u);
        tc::mma_commit(empty + stage);
        if (b + C::SUB >= b1) tc::mma_commit(acc_full);
      }
      __syncwarp();
      if (++stage == C::STAGES) { stage = 0; phase ^= 1u; }
    }
  } else {
    // lane base + lane is a layer row, a TMEM column a token
    const int lane_base = (warp & 3) * 32;
    const int row = r0 + lane_base + lane;
    if (tc::mbar_wait_warp(acc_full, 0, abort_flag, p.wait_limit)) {
      tc::fence_after_sync();
      float* part = reinterpret_cast<float*>(smem);      // [token][128 rows]; the ring is empty
      for (int c = 0; c < p.M; c += 16) {
        uint32_t v[16];
        tc::tmem_ld_32x16(tmem_base + (uint32_t(lane_base) << 16) + uint32_t(c), v);
        tc::tmem_ld_wait();
        if (splits == 1) {
          T* y = static_cast<T*>(p.Y) + int64_t(c) * p.ldy + row;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (row < p.R && c + i < p.M) y[i * p.ldy] = from_f32<T>(__uint_as_float(v[i]));
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) part[(c + i) * 128 + lane_base + lane] = __uint_as_float(v[i]);
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (splits > 1) {
    // every CTA of the cluster sums its share of the tokens, the splits in order
    tc::cluster_sync();
    // (a warp a token, a lane four layer rows, all loads before the first sum)
    const int row = r0 + 4 * lane;
    for (int t = split + splits * warp; t < p.M; t += splits * (FEW_THREADS / 32)) {
      const uint32_t at = tc::smem_u32(smem + (t * 128 + 4 * lane) * 4);
      float4 part[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < splits) part[q] = tc::ld_cluster_f32x4(tc::map_cluster(at, uint32_t(q)));
      float4 v = part[0];
#pragma unroll
      for (int q = 1; q < 8; ++q)
        if (q < splits) {
          v.x += part[q].x;
          v.y += part[q].y;
          v.z += part[q].z;
          v.w += part[q].w;
        }
      T* y = static_cast<T*>(p.Y) + int64_t(t) * p.ldy + row;
      const float o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row + i < p.R) y[i] = from_f32<T>(o[i]);
    }
    __syncwarp();
    // No CTA leaves while its partial sums are read.  An execution barrier is enough: the first
    // lane of a warp has a layer row (r0 < R) and stores what the whole warp's load brought, so
    // every load has arrived before its warp does.
    tc::cluster_sync_relaxed();
  }
  if (*abort_flag) {
    if (warp == 0 && lane == 0) tc::drain_tma_ring(full, C::STAGES, issued);
    if (warp == 1) {                 // by the lane that issued the MMAs
      if (tc::elect_one()) {
        tc::mma_commit(drain);
        tc::mbar_drain(drain, 0);
      }
      __syncwarp();
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

// ------------------------------------------------------------------ many tokens
// A pair of CTAs computes 256 layer rows x bn tokens: rank r loads layer rows r0 + 128 r ..
// and tokens n0 + bn/2 r .. (its halves of the operands), the scales of its layer rows and of
// all of the tile's tokens; rank 0 issues the MMAs.  The accumulator rows r0 + 128 r .. land
// in rank r's TMEM.  8 epilogue warps per CTA take the whole tile into registers and release
// the accumulator before they convert and store.  Up to 128 tokens two accumulators alternate,
// so that the next tile's MMAs do not wait for that; two of more and the scales do not fit the
// 512 TMEM columns, and each tile then starts about 2000 cycles after the last.
namespace pair {

// A stage of the ring is two boxes, 512 columns: each stage costs the issuing warp about 400
// cycles of waiting, committing and looping whatever it holds, which one box's MMAs hide at 256
// tokens only (256 cycles at 128 tokens).  The ring's shape goes with the token tile.
constexpr int SUB = 2;                            // boxes of a stage
constexpr int MAX_STAGES = 5;
constexpr int MAX_SPLITS = 4;                     // pairs that share a tile's K
constexpr int RING = 222 * 1024;                  // bytes of shared memory for the stages
constexpr int SMEM = RING + 1024 /*align*/ + 256 /*barriers*/;
constexpr int NB = 2;                             // scale tiles that a token tile touches at most
constexpr int THREADS = 320;
constexpr int GROUP = 16;                         // token tiles per group of the tile order

// Byte offsets in a stage: W's boxes first, then X's, then the scales of W and of X.
__host__ __device__ constexpr int x_off() { return SUB * A_BOX; }
__host__ __device__ constexpr int s_off(int bn) { return x_off() + SUB * (bn / 2) * KB; }
__host__ __device__ constexpr int stage_bytes(int bn, int nb) { return s_off(bn) + SUB * 1024 * (1 + nb); }
__host__ __device__ constexpr int sf_cols(int nb) { return SUB * 8 * (1 + nb); }
__host__ __device__ constexpr int tile_nb(int bn) { return (bn + 127) / 128; }   // 64 and 192 tokens
                                                  // start on either half of a scale tile
__host__ __device__ constexpr int stages_of(int bn) {
  return RING / stage_bytes(bn, tile_nb(bn)) < MAX_STAGES ? RING / stage_bytes(bn, tile_nb(bn)) : MAX_STAGES;
}
__host__ __device__ constexpr int accs_of(int bn) { return bn <= 128 ? 2 : 1; }
constexpr bool fits(int bn) {
  return bn * 512 <= RING &&
         accs_of(bn) * bn + stages_of(bn) * sf_cols(tile_nb(bn)) <= 512 && stages_of(bn) >= 3 &&
         stage_bytes(bn, tile_nb(bn)) % 1024 == 0;
}
static_assert(fits(64) && fits(128) && fits(192) && fits(256), "TMEM, shared memory");

// t-th tile: groups of GROUP token tiles, row tile by row tile inside a group, so that the
// tiles in flight together share operand rows in L2
__device__ __forceinline__ void tile_of(const Prob& p, int t, int& r0, int& n0) {
  const int per = GROUP * p.ntr;
  const int g = t / per, q = t - g * per;
  const int w = min(GROUP, p.ntt - g * GROUP);
  r0 = q / w * 256;
  n0 = (g * GROUP + q % w) * p.bn;
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 1)
k_mx_pair(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
          const __grid_constant__ CUtensorMap wsmap, const __grid_constant__ CUtensorMap xsmap,
          Prob p, uint32_t idesc, int32_t* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + RING);
  uint64_t* empty = full + MAX_STAGES;
  uint64_t* acc_full = empty + MAX_STAGES;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* issued_slot = tmem_slot + 2;          // the partner's fill count (abort path)

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  // a cluster is one pair, or the pairs that share a tile's K (one tile per cluster then)
  const uint32_t base = tc::cluster_rank() & ~1u, rank = tc::cluster_rank() & 1u;
  const int split = int(base >> 1), splits = int(tc::cluster_size() >> 1);
  const int pair_id = int(blockIdx.x) / (2 * splits), n_pairs = int(gridDim.x) / (2 * splits);
  const int tiles = p.ntr * p.ntt;
  const int nk = (p.boxes + SUB - 1) / SUB;       // stages along K; this pair's: k0 .. k1 - 1
  const int k0 = int(int64_t(nk) * split / splits), k1 = int(int64_t(nk) * (split + 1) / splits);
  const int stages = p.stages, bytes = stage_bytes(p.bn, p.nb), cols = sf_cols(p.nb);
  const uint32_t sf_base = 512 - uint32_t(stages * cols);      // TMEM columns below: accumulators

  if (threadIdx.x == 64) {
    tc::prefetch_map(&wmap);
    tc::prefetch_map(&xmap);
    tc::prefetch_map(&wsmap);
    tc::prefetch_map(&xsmap);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < MAX_STAGES; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(acc_full + i, 1);
      tc::mbar_init(acc_empty + i, 16);           // 8 epilogue warps of each CTA
    }
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    *issued_slot = 0;
    tc::fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(tmem_slot, 512);
    tc::tmem_relinquish_pair();
  }
  tc::fence_before_sync();
  tc::cluster_sync();                             // both CTAs' barriers and TMEM ready
  tc::fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const uint16_t both = uint16_t(0x3u << base);   // the pair's CTAs in the cluster
  const uint32_t peer_flag = tc::cluster_addr(const_cast<int*>(abort_flag), base + (rank ^ 1u));
  int64_t issued = 0;

  // one fill: boxes past the tensors' ends read as zeros and count in full
  const auto load = [&](int stage, int k, int r0, int n0) {
    uint8_t* a = smem + stage * bytes;
    uint8_t* x = a + x_off();
    uint8_t* s = a + s_off(p.bn);
    if (rank == 0) tc::mbar_expect_tx(full + stage, 2 * uint32_t(bytes));
    const uint32_t cbar = tc::cluster_addr(full + stage, base);
    const int ra = r0 + 128 * int(rank), rx = n0 + p.bn / 2 * int(rank);
#pragma unroll
    for (int j = 0; j < SUB; ++j) {
      tc::tma_load_2d_pair(a + j * A_BOX, &wmap, (SUB * k + j) * KB, ra, cbar);
      tc::tma_load_2d_pair(x + j * (p.bn / 2 * KB), &xmap, (SUB * k + j) * KB, rx, cbar);
    }
    tc::tma_load_2d_pair(s, &wsmap, k * 256, r0 / 128 + int(rank), cbar);
    tc::tma_load_2d_pair(s + SUB * 1024, &xsmap, k * 256, n0 / 128, cbar);
  };
  const auto wait = [&](uint64_t* bar, uint32_t parity, bool cluster_scope = false, bool give_up = false) {
    return tc::mbar_wait_pair_warp(bar, parity, abort_flag, peer_flag, give_up ? 0u : p.wait_limit,
                                   cluster_scope);
  };

  allow_successor();
  wait_for_predecessor();
  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = pair_id; t < tiles && ok; t += n_pairs) {
      int r0, n0;
      tile_of(p, t, r0, n0);
      for (int k = k0; k < k1; ++k) {
        if (!wait(empty + stage, phase ^ 1u)) { ok = false; break; }
        if (tc::elect_one()) load(stage, k, r0, n0);
        __syncwarp();
        ++issued;
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
    }
    // every fill consumed: the MMAs' last arrivals on this CTA's empty barriers have landed
    // before the CTA can exit
    if (ok)
      for (int st = 0; st < stages; ++st) {
        const int64_t n = issued / stages + (st < issued % stages ? 1 : 0);
        if (n > 0 && !wait(empty + st, uint32_t((n - 1) & 1))) break;
      }
  } else if (warp == 1) {
    if (rank == 0) {
      int stage = 0;
      uint32_t phase = 0;
      AccRing ring(p.accs);
      bool ok = true;
      const uint64_t adesc0 = tc::smem_desc_sw128(smem, 16, 1024);
      const uint64_t sdesc0 = tc::smem_desc_rows16(smem + s_off(p.bn));
      const int last = p.give_up >= 0 && split == splits - 1 ? k0 + p.give_up : k1;
      const uint32_t xbox = uint32_t(p.bn / 2 * KB) >> 4;       // descriptors count in 16 bytes
      const uint32_t tile_cols = 4 * uint32_t(p.nb);            // TMEM columns of 128 columns' scales of X
      for (int t = pair_id; t < tiles && ok; t += n_pairs) {
        int r0, n0;
        tile_of(p, t, r0, n0);
        // a token tile may start in the middle of a scale tile, 32 tokens to a TMEM column; the
        // MMA takes its scales from an even column only, so tiles are multiples of 64 tokens
        const uint32_t first = uint32_t((n0 & 64) >> 5);
        if (!wait(acc_empty + ring.at, ring.phase ^ 1u, true)) { ok = false; break; }
        const uint32_t d = tmem_base + uint32_t(ring.at * p.bn);
        tc::fence_after_sync();
        for (int k = k0; k < k1; ++k) {
          if (!wait(full + stage, phase, false, k >= last)) { ok = false; break; }
          tc::fence_after_sync();
          const uint64_t ad = adesc0 + uint32_t(stage * (bytes >> 4));
          const uint64_t xd = ad + (x_off() >> 4);
          const uint64_t sd = sdesc0 + uint32_t(stage * (bytes >> 4));
          const uint32_t sfa = tmem_base + sf_base + uint32_t(stage * cols);
          const uint32_t sfb = sfa + 8 * SUB;
          const int todo = p.steps - 4 * SUB * k;
          if (tc::elect_one()) {
#pragma unroll
            for (int h = 0; h < 2 * SUB; ++h) {
              tc::copy_scales_pair(sfa + 4 * h, sd + 32 * h);
#pragma unroll
              for (int j = 0; j < NB; ++j)
                if (j < p.nb)
                  tc::copy_scales_pair(sfb + tile_cols * h + 4 * j, sd + 64 * SUB * (1 + j) + 32 * h);
            }
#pragma unroll
            for (int kk = 0; kk < 4 * SUB; ++kk)
              if (kk < todo)
                tc::mma_mxf4_pair(d, ad + (kk >> 2) * (A_BOX >> 4) + 2 * (kk & 3),
                                  xd + (kk >> 2) * xbox + 2 * (kk & 3),
                                  idesc | ((kk & 1) ? ODD_HALF : 0u), sfa + 4 * (kk >> 1),
                                  sfb + first + tile_cols * (kk >> 1), (k > k0 || kk > 0) ? 1u : 0u);
            tc::mma_commit_pair(empty + stage, both);
            if (k + 1 == k1) tc::mma_commit_pair(acc_full + ring.at, both);
          }
          __syncwarp();
          if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        ring.next();
      }
      // every accumulator handed back: rank 1's last arrivals have landed in this CTA's shared
      // memory before it can exit (they arrive before they store, so no store is waited for)
      if (ok)
        for (int i = 0; i < p.accs; ++i)
          if (!wait(acc_empty + i, ring.last(i), true)) break;
    }
  } else {
    const int lane_base = (warp & 3) * 32;
    const int half = p.bn / 2, c0 = ((warp - 2) >> 2) * half;     // this warp's tokens of the tile
    const uint32_t acc_empty0 = tc::cluster_addr(acc_empty, base);
    AccRing ring(p.accs);
    for (int t = pair_id; t < tiles; t += n_pairs) {
      int r0, n0;
      tile_of(p, t, r0, n0);
      if (!wait(acc_full + ring.at, ring.phase)) break;
      tc::fence_after_sync();
      uint32_t v[4][32];
      const uint32_t at = tmem_base + (uint32_t(lane_base) << 16) + uint32_t(ring.at * p.bn + c0);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (32 * c < half) tc::tmem_ld_32x32(at + 32 * c, v[c]);
      tc::tmem_ld_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster_relaxed(acc_empty0 + uint32_t(ring.at * 8));
      ring.next();
      const int row = r0 + 128 * int(rank) + lane_base + lane;
      if (splits > 1) {
        // this pair's partial sums, [token][128 rows]; every load into the ring was consumed
        float* part = reinterpret_cast<float*>(smem) + c0 * 128 + lane_base + lane;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (32 * c < half) {
#pragma unroll
            for (int i = 0; i < 32; ++i) part[(32 * c + i) * 128] = __uint_as_float(v[c][i]);
          }
      } else if (row < p.R) {
        const int live = min(half, p.M - n0 - c0);
        T* y = static_cast<T*>(p.Y) + int64_t(n0 + c0) * p.ldy + row;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (32 * c + 32 <= live) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              *y = from_f32<T>(__uint_as_float(v[c][i]));
              y += p.ldy;
            }
          } else if (32 * c < live) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (32 * c + i < live) *y = from_f32<T>(__uint_as_float(v[c][i]));
              y += p.ldy;
            }
          }
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (splits > 1) {
    // an abort is the whole cluster's: the barriers below are
    if (threadIdx.x == 0 && *abort_flag) {
      for (int q = 0; q < 2 * splits; ++q)
        tc::st_cluster_u32(tc::cluster_addr(const_cast<int*>(abort_flag), uint32_t(q)), 1u);
      asm volatile("fence.acq_rel.cluster;" ::: "memory");
    }
    __syncwarp();
    tc::cluster_sync();        // the partial sums are written
    if (!*abort_flag) {
      // every pair sums its share of the tokens, the splits in order (a warp a token, a lane
      // four layer rows, all loads before the first sum)
      int r0, n0;
      tile_of(p, pair_id, r0, n0);
      // (no load is left in flight when the CTAs part: a CTA whose layer rows do not exist makes
      // none, the others' results are stored by their first lanes at least)
      const int row = r0 + 128 * int(rank) + 4 * lane;
      const int live = r0 + 128 * int(rank) < p.R ? min(p.bn, p.M - n0) : 0;
      for (int t = split + splits * warp; t < live; t += splits * (THREADS / 32)) {
        const uint32_t at = tc::smem_u32(smem + (t * 128 + 4 * lane) * 4);
        float4 part[MAX_SPLITS];
#pragma unroll
        for (int q = 0; q < MAX_SPLITS; ++q)
          if (q < splits) part[q] = tc::ld_cluster_f32x4(tc::map_cluster(at, uint32_t(2 * q) + rank));
        float4 v = part[0];
#pragma unroll
        for (int q = 1; q < MAX_SPLITS; ++q)
          if (q < splits) {
            v.x += part[q].x;
            v.y += part[q].y;
            v.z += part[q].z;
            v.w += part[q].w;
          }
        T* y = static_cast<T*>(p.Y) + int64_t(n0 + t) * p.ldy + row;
        const float o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row + i < p.R) y[i] = from_f32<T>(o[i]);
      }
    }
    __syncwarp();
  }
  tc::cluster_sync_relaxed();  // all CTAs out of their loops: the abort flags are final
  if (*abort_flag) {
    // A wait gave up in one of the CTAs, which raised both flags.  (1) rank 0's MMAs land, and
    // in both CTAs the arrival behind all those that they made there; (2) the producers
    // exchange their fill counts and the one behind fills the phases the other filled (boxes at
    // the origin), so every phase of rank 0's full barriers that either CTA loaded into
    // completes; (3) rank 0 waits for them, i.e. for both CTAs' copies; (4) neither CTA exits
    // before that.
    if (warp == 1) {
      if (tc::elect_one()) {
        if (rank == 0) tc::mma_commit_pair(drain, both);    // by the lane that issued the MMAs
        tc::mbar_drain(drain, 0);
      }
      __syncwarp();
    }
    if (warp == 0 && lane == 0)
      tc::st_cluster_u32(tc::cluster_addr(issued_slot, base + (rank ^ 1u)), uint32_t(issued));
    tc::fence_before_sync();
    tc::cluster_sync();
    if (warp == 0 && lane == 0) {
      const int64_t other = int64_t(*issued_slot);
      for (int64_t f = issued; f < other; ++f) load(int(f % stages), 0, 0, 0);
      if (rank == 0) tc::drain_tma_ring(full, stages, other > issued ? other : issued);
    }
    tc::fence_before_sync();
    tc::cluster_sync();
    if (threadIdx.x == 0 && rank == 0) raise_status(status, GPTQ_ERR_TIMEOUT);
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace pair

// ------------------------------------------------------------------ host
// rows of `row_bytes` bytes of codes, boxes of 128 bytes x box_rows
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

// scale tiles as rows (128 matrix rows) of ct * 512 bytes, boxes of four tiles x box_rows;
// tiles past the ends read as zeros
bool encode_scales(CUtensorMap* m, const uint8_t* scales, uint64_t ct, uint64_t tile_rows,
                   uint32_t box_rows) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {ct * 64, tile_rows};
  const cuuint64_t strides[1] = {ct * 512};
  const cuuint32_t box[2] = {256, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_INT64, 2, const_cast<uint8_t*>(scales), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of CTAs that fill an SM each that run at once, to choose a split of K by: SMs come in
// groups whose size is no multiple of 4 or 8.  A share of the SMs, just below what the occupancy
// query gives (of 148 SMs 74, 32 and 14 clusters of 2, 4 and 8 for 74, 33 and 15): a split that
// is one cluster too many costs a second wave, one that is not taken some of its gain.
int64_t clusters_at_once(int ctas, int sms) {
  return ctas <= 2 ? sms / ctas : ctas <= 4 ? sms * 2 / 9 : sms / 10;
}

cudaLaunchConfig_t cluster_launch(unsigned ctas, int cluster, int threads, int smem,
                                  cudaStream_t st, cudaLaunchAttribute (&at)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(cluster);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1] = may_start_early();
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cfg;
}

template <int BN, typename T>
gptq_status launch_few(cudaStream_t st, const uint32_t* xc, const uint32_t* wc, uint64_t row_bytes,
                       const Prob& p, int sms, int32_t* status) {
  using C = Few<BN>;
  CUtensorMap wmap, xmap;
  if (!encode_codes(&wmap, wc, row_bytes, uint64_t(p.R), 128) ||
      !encode_codes(&xmap, xc, row_bytes, uint64_t(p.M), BN))
    return GPTQ_ERR_UNSUPPORTED;
  const int rows = (p.R + 127) / 128;
  int splits = 1;
  while (splits < 8 && rows <= clusters_at_once(2 * splits, sms) && p.boxes >= 2 * C::SUB * splits)
    splits *= 2;
  GPTQ_CUDA(allow_smem(k_mx_few<BN, T>, C::SMEM));
  cudaLaunchAttribute at[2];
  const cudaLaunchConfig_t cfg = cluster_launch(unsigned(rows * splits), splits, FEW_THREADS,
                                                C::SMEM, st, at);
  GPTQ_LAUNCHED(cudaLaunchKernelEx(&cfg, k_mx_few<BN, T>, wmap, xmap, p, status), "k_mx_few");
  return GPTQ_OK;
}

template <typename T>
gptq_status launch_pair(cudaStream_t st, const uint32_t* xc, const uint32_t* wc, uint64_t row_bytes,
                        const Prob& p, int splits, int sms, int32_t* status) {
  CUtensorMap wmap, xmap, wsmap, xsmap;
  if (!encode_codes(&wmap, wc, row_bytes, uint64_t(p.R), 128) ||
      !encode_codes(&xmap, xc, row_bytes, uint64_t(p.M), uint32_t(p.bn / 2)) ||
      !encode_scales(&wsmap, p.ws, uint64_t(p.ct), uint64_t((p.R + 127) / 128), 1) ||
      !encode_scales(&xsmap, p.xs, uint64_t(p.ct), uint64_t((p.M + 127) / 128), uint32_t(p.nb)))
    return GPTQ_ERR_UNSUPPORTED;
  GPTQ_CUDA(allow_smem(pair::k_mx_pair<T>, pair::SMEM));
  const int clusters = int(std::min<int64_t>(sms / (2 * splits), int64_t(p.ntr) * p.ntt));
  cudaLaunchAttribute at[2];
  const cudaLaunchConfig_t cfg = cluster_launch(unsigned(2 * splits * clusters), 2 * splits,
                                                pair::THREADS, pair::SMEM, st, at);
  GPTQ_LAUNCHED(cudaLaunchKernelEx(&cfg, pair::k_mx_pair<T>, wmap, xmap, wsmap, xsmap, p,
                                   idesc_of(256, p.bn), status), "k_mx_pair");
  return GPTQ_OK;
}

template <typename T>
gptq_status by_tokens(cudaStream_t st, const uint32_t* xc, const uint32_t* wc, uint64_t row_bytes,
                      Prob p, int sms, int32_t* status) {
  // K split over clusters where there are few tokens or few layer rows.  Measured (few tokens'
  // kernel against pairs, us): 16 tokens 4096 x 11008 6.4 / 11.9, 49152 x 12288 55.7 / 53.9; 64
  // tokens 4096 x 11008 7.9 / 12.2, 5120 x 5120 7.7 / 7.8, 11008 x 4096 8.3 / 7.2, 49152 x 12288
  // 64.9 / 54.0; 128 tokens 12288 x 12288 21.7 / 14.2.  Up to 32 tokens the pairs, whose least
  // tile is 64 of them, win on the widest layers only, by 3%: there the rule has no exception.
  p.ntr = (p.R + 255) / 256;
  if (p.M <= 16) return launch_few<16, T>(st, xc, wc, row_bytes, p, sms, status);
  if (p.M <= 32) return launch_few<32, T>(st, xc, wc, row_bytes, p, sms, status);
  if (p.M <= 64 && 4 * p.ntr <= sms) return launch_few<64, T>(st, xc, wc, row_bytes, p, sms, status);
  // the token tile, and the pairs that share its K, by the time of the pairs' waves in cycles: a
  // step takes about 64 + bn/4 (operand bytes into shared memory: 4 KB of W, bn/64 KB of X), a
  // tile of a single accumulator starts late, partial sums are written and read again
  int64_t best = 0;
  int splits = 1;
  const int64_t pairs = sms / 2;
  const int nk = (p.boxes + pair::SUB - 1) / pair::SUB;
  for (int bn = 256; bn >= 64; bn -= 64) {
    const int64_t tiles = int64_t(p.ntr) * ((p.M + bn - 1) / bn);
    for (int s = 1; s <= pair::MAX_SPLITS && (s == 1 || (tiles <= clusters_at_once(2 * s, sms) && nk >= 2 * s)); s *= 2) {
      const int64_t steps = s == 1 ? p.steps : int64_t((nk + s - 1) / s) * 4 * pair::SUB;
      const int64_t time = (tiles * s + pairs - 1) / pairs * (steps * (64 + bn / 4) + (pair::accs_of(bn) == 1 ? 2000 : 200)) +
                           (s > 1 ? 1500 + 8 * bn : 0);
      if (best == 0 || time < best) { best = time; p.bn = bn; splits = s; }
    }
  }
  p.accs = pair::accs_of(p.bn);
  p.nb = pair::tile_nb(p.bn);
  p.stages = pair::stages_of(p.bn);
  p.ntt = (p.M + p.bn - 1) / p.bn;
  return launch_pair<T>(st, xc, wc, row_bytes, p, splits, sms, status);
}

}  // namespace

gptq_status mx_matmul_run(cudaStream_t st, const uint32_t* xc, const uint8_t* xs, int M,
                          const uint32_t* wc, const uint8_t* ws, int R, int C, void* Y, int dt,
                          int64_t ldy, int32_t* status) {
  const int sms = sm_count();
  if (sms <= 0) return GPTQ_ERR_CUDA;
  const int nb = (C + 31) / 32;
  Prob p = {};
  p.xs = xs;
  p.ws = ws;
  p.Y = Y;
  p.ldy = ldy;
  p.M = M;
  p.R = R;
  p.steps = (nb + 1) / 2;
  p.ct = (nb + 3) / 4;
  p.boxes = (nb + 7) / 8;
  p.wait_limit = pipeline_wait_limit();
  p.give_up = int(std::min<int64_t>(mx_give_up(), p.boxes));
  const uint64_t row_bytes = uint64_t(nb) * 16;
  switch (dt) {
    case GPTQ_F32: return by_tokens<float>(st, xc, wc, row_bytes, p, sms, status);
    case GPTQ_F16: return by_tokens<__half>(st, xc, wc, row_bytes, p, sms, status);
    default: return by_tokens<__nv_bfloat16>(st, xc, wc, row_bytes, p, sms, status);
  }
}

}  // namespace gptq
