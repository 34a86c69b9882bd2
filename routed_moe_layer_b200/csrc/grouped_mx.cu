// Grouped products of MX operands (mx_format.cuh) on the sm_100a tensor cores:
// for every row r of group e
//   D[r, n] = sum_b 2^(pa[r,b] + pw[e,n,b]) * sum_{k in block b} a[r,k] * w[e,n,k]
// with the block-scaled tcgen05.mma, which reads 8- or 4-bit elements from
// shared memory and their scales from TMEM and accumulates in fp32, and two
// ends:
//   MX_ROWS    out[dest(r), n] = bf16( row_w[r] * D[r, n] )   (dest(r) = r, row_w = 1
//              where they are not given)
//   MX_SWIGLU  h[r, i] = silu(D[r, i]) * D[r, I + i], quantised in the format of the
//              operands: 32 columns of a row are one block, which one epilogue
//              thread holds in registers, so h never exists in a wider type.
//
// Shape: persistent clusters of two CTAs share one pair MMA (cta_group::2) of
// 256 rows x 256 columns; a K step is 128 bytes of every row: 128 elements
// (MXFP8, 4 MMAs of K = 32) or 256 (MXFP4, 4 MMAs of K = 64).  Bytes a step and
// MMA time a step are those of the bf16 kernel (grouped_gemm.cu), for two and
// four times the elements.  Each CTA loads its 128 rows of A and half of the B
// tile, its own rows' scales of A and all 256 columns' scales of B.
// tcgen05.cp wants the scale words of 128 operand rows as 32 rows of 16 bytes,
// row l holding those of operand rows l, l+32, l+64, l+96.  B's rows are laid
// in shared memory so that this is the order of its words in memory: operand
// row j*32 + l is matrix row 4l + j (four TMA boxes of every fourth row), one
// TMA copy then brings 128 words as they are, and the epilogue reads
// accumulator column j*32 + l as output column 4l + j.  A's tiles start at any
// row, which TMA does not take for 4-byte words: a warp loads them and writes
// them to shared memory in that order, 16 words a row (2048 elements) at a
// time, because the proxy fence and the release across the pair that this
// takes cost 1 us when they are paid in every K step.
// Warp roles (both CTAs):
//   warp 0       TMA loads of A and of B's scales (counted on the leader CTA's
//                barrier)
//   warp 1       TMEM; in the leader it copies the scales to TMEM and issues the
//                MMAs
//   warp 2       TMA loads of B
//   warp 3       scales of A
//   warps 4..19  epilogue: four warps per TMEM lane quarter, 64 accumulator
//                columns a thread (eight warps of 128 columns were bound by their
//                own latency, and left no registers for the rest)
// TMEM: columns 0..255 the accumulator, 256 + 32 s.. the scales of stage s.
// The accumulator is not double-buffered (two of them leave no columns for the
// scales); the epilogue reads it whole into registers and hands it back before
// it computes or stores anything.
// Every wait is bounded (common.cuh).
//
// What bounds it: at 155,296 rows and back to back the card's 1,000 W (SM clock
// 1.28 to 1.46 GHz).  MXFP8 K = 2048, N = 1536: 543 us (1.80 PFLOP/s; one launch
// on a cool card 440), of which the MMAs alone would take 363 and the loads
// alone 280; MXFP4 302 us (3.2 PFLOP/s; 251), 189 and 156.  MXFP8 K = 768, N = 2048:
// 325 us (275) for 636 MB of output, which alone take 163 us at the 3.9 TB/s that
// writes reach.
#include "mx_mma.cuh"

namespace rmoe {

namespace {

constexpr int BM = 128;          // rows per CTA
constexpr int TILE_M = 2 * BM;   // rows per pair tile
constexpr int BN = 256;          // accumulator columns
constexpr int KB = 128;          // bytes of a row per K step
constexpr int MAX_STAGES = 6;
constexpr int A_BYTES = BM * KB;
constexpr int B_BYTES = BN / 2 * KB;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int B_BOX = 32;        // B rows per TMA box (every fourth row of the matrix)
constexpr int SF_BYTES = MX_SF_BYTES;
constexpr int THREADS = 640;
constexpr int EPI_WARP0 = 4;
constexpr int EPI_WARPS = 16;
constexpr int EPI_COLS = 64;     // accumulator columns of an epilogue thread
constexpr int OUT_PITCH = BN * 2 + 16;  // bytes of an output row in shared memory (no conflicts)
constexpr int SFA_WORDS = 16;    // words per row in a buffer of A's scales
constexpr int SFA_BYTES = SFA_WORDS * SF_BYTES;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TMEM_SF = 256;        // + 32 per stage: A, 4 per word, ...
constexpr uint32_t TMEM_SFB = 8;         // ... B, 8 per word, 4 per half

template <int FMT, int EPI>
struct Shape {
  static constexpr int kWords = FMT == MOE_MXFP8 ? 1 : 2;  // scale words per row and K step
  static constexpr int kStages = EPI == MX_ROWS ? 4 : 6;   // rows: room for the output tile
  static constexpr int kSfb = kWords * 2 * SF_BYTES;       // B's scales, both halves
  static constexpr int kOffSfb = kStages * STAGE_BYTES;
  static constexpr int kOffSfa = kOffSfb + kStages * kSfb;
  static constexpr int kOffOut = kOffSfa + 2 * SFA_BYTES;
  static constexpr int kOffTail = kOffOut + (EPI == MX_ROWS ? BM * OUT_PITCH : 0);
};

struct __align__(8) SmemTail {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t sfa_full[2];
  uint64_t sfa_empty[2];
  uint64_t tfull;
  uint64_t tempty;
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  MxGroups groups;
};

// Block-scaled pair MMA.  Element and scale formats in idesc: A and B E4M3
// with one scale per 32 of K = 32 (MXFP8), or E2M1 with two of K = 64 (MXFP4).
template <int FMT>
__device__ __forceinline__ void umma_mx_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (FMT == MOE_MXFP8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// 32 rows of 16 bytes to 4 TMEM columns, repeated in the four lane quarters, in
// both CTAs of the pair from the same shared-memory offset.
__device__ __forceinline__ void tmem_copy_sf_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
               : "memory");
}

// Tile loads to a shared-memory address, completion counted on the barrier at
// cluster address mbar (the leader's).
__device__ __forceinline__ void tma_load_2d_at(uint32_t dst, const CUtensorMap* map, uint32_t mbar,
                                               int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d_at(uint32_t dst, const CUtensorMap* map, uint32_t mbar,
                                               int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Arrive on a barrier of the cluster, releasing this thread's shared-memory
// writes (and those of the warp's lanes before a __syncwarp) to its CTAs.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// Acquires at cluster scope a phase that mbar_wait has seen complete.
__device__ __forceinline__ void mbar_acquire_cluster(uint64_t* bar, uint32_t parity) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t}\n" ::"r"(
          smem_u32(bar)),
      "r"(parity)
      : "memory");
}

// 32 TMEM lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

// Accumulator columns of epilogue part 0..3: 64 output columns part*64.. (MX_ROWS),
// or gate and up of output columns part*32.. (MX_SWIGLU).  Output column 4l + j
// of a 128-column half lies at j*32 + l.
template <int EPI>
__device__ __forceinline__ void load_part(uint32_t tb, int part, uint32_t (&v)[EPI_COLS]) {
  if constexpr (EPI == MX_ROWS) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      tmem_ld_32x32b_x16(tb + (part >> 1) * 128 + 32 * j + (part & 1) * 16,
                         *reinterpret_cast<uint32_t(*)[16]>(v + 16 * j));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      tmem_ld_32x32b_x8(tb + 32 * j + part * 8, *reinterpret_cast<uint32_t(*)[8]>(v + 8 * j));
      tmem_ld_32x32b_x8(tb + BN / 2 + 32 * j + part * 8,
                        *reinterpret_cast<uint32_t(*)[8]>(v + 32 + 8 * j));
    }
  }
  tmem_ld_wait();
}

// Whether a tile's wait has come to its end in all the epilogue warps that work
// together (MX_ROWS: those of a quarter, which share barriers): they leave the
// tile loop together when it has run out in one.
template <int EPI>
__device__ __forceinline__ bool epilogue_agrees(int q, bool ok) {
  if constexpr (EPI == MX_SWIGLU) return ok;
  return warps_agree<4>(q + 1, ok);
}

// t: this CTA's part of the tile; out: the tile's rows in shared memory (MX_ROWS).
template <int FMT, int EPI>
__device__ __forceinline__ void store_part(const MxGemmArgs& a, const uint32_t (&v)[EPI_COLS],
                                           const Tile& t, int r_in_tile, int part, uint32_t out) {
  const int row = t.row0 + r_in_tile;
  if constexpr (EPI == MX_ROWS) {
    // The tile goes to shared memory and from there, a row's 256 columns at a
    // time, by bulk copies.  Stores from registers (64 KB a tile and SM, more
    // than the SM's path to L2 takes at once) queue up in front of the MMA
    // warp's barriers: its K steps then took 500 cycles to issue, not 200.
    const int lane = r_in_tile & 31, q = r_in_tile >> 5;
    const float w = a.row_w && r_in_tile < t.rows ? a.row_w[row] : 1.0f;
    // this lane's row of the copies: 8 rows a warp
    const int crow = q * 32 + part * 8 + lane;
    int dest = -1;
    if (lane < 8 && crow < t.rows) {
      dest = a.row_dest ? a.row_dest[t.row0 + crow] : t.row0 + crow;
      if (dest >= a.out_rows) dest = -1;
    }
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last tile's copies
    warps_sync<4>(q + 1);
#pragma unroll
    for (int k = 0; k < EPI_COLS / 8; ++k) {
      uint32_t pk[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 8 * k + 2 * i;
        pk[i] = pack_bf16x2(w * __uint_as_float(v[(n & 3) * 16 + (n >> 2)]),
                            w * __uint_as_float(v[((n + 1) & 3) * 16 + (n >> 2)]));
      }
      st_shared_v4(out + r_in_tile * OUT_PITCH + part * (EPI_COLS * 2) + 16 * k, pk);
    }
    fence_proxy_async_smem();  // these writes -> the copies
    warps_sync<4>(q + 1);
    if (dest >= 0)
      bulk_store(static_cast<__nv_bfloat16*>(a.out) + (size_t)dest * a.n_valid + t.nt * BN,
                 out + crow * OUT_PITCH, 2 * min(BN, a.n_valid - t.nt * BN));
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  } else {
    if (r_in_tile >= t.rows) return;
    // one block of h: 32 columns of the row
    const int col0 = t.nt * (BN / 2) + part * MX_BLOCK;
    uint32_t byte = 0;  // a word's bytes past the last column's block are 0
    if (col0 < a.n_valid) {
      float h[MX_BLOCK];
      uint32_t m = 0;
#pragma unroll
      for (int n = 0; n < MX_BLOCK; ++n) {
        const int c = (n & 3) * 8 + (n >> 2);
        h[n] = silu_f(__uint_as_float(v[c])) * __uint_as_float(v[32 + c]);
        m = max(m, __float_as_uint(h[n]) & 0x7fffffffu);
      }
      byte = mx_scale_byte<FMT>(m);
      uint32_t q[8];
      mx_encode<FMT>(h, byte, q);
      uint8_t* dst =
          static_cast<uint8_t*>(a.out) + ((size_t)row * a.n_valid + col0) / MxFmt<FMT>::kPerByte;
      if constexpr (FMT == MOE_MXFP8)
        st_global_v8(dst, q);
      else
        *reinterpret_cast<uint4*>(dst) = make_uint4(q[0], q[1], q[2], q[3]);
    }
    reinterpret_cast<uint8_t*>(a.out_scales + (size_t)t.nt * a.rows + row)[part] =
        static_cast<uint8_t>(byte);
  }
}

template <int FMT, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    grouped_mx_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmSB, const MxGemmArgs args) {
  using S = Shape<FMT, EPI>;
  constexpr int STAGES = S::kStages;
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ __align__(1024) uint8_t smem[];
  SmemTail& st = *reinterpret_cast<SmemTail*>(smem + S::kOffTail);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&st.full[s], 1);   // leader: its producer's expect-tx arrive
      mbar_init(&st.empty[s], 1);  // both: one commit from the leader's MMA thread
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&st.sfa_full[b], 2);   // leader: the scale warps of both CTAs
      mbar_init(&st.sfa_empty[b], 1);  // both: one commit
    }
    mbar_init(&st.tfull, 1);
    mbar_init(&st.tempty, 2 * EPI_WARPS);  // leader: every epilogue warp of both CTAs
    mbar_init(&st.drain, 1);
    st.abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSB);
  }
  const int total = mx_group_table<TILE_M>(args, st.groups) * args.n_tiles;
  if (cluster >= total) return;  // the same for both CTAs of the cluster; nothing allocated yet
  cluster_sync();                // both CTAs' barriers exist before any cross-CTA traffic

  if (warp == 1) {
    tmem_alloc_pair(&st.tmem_base, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = uniform(st.tmem_base);
  const WaitCtx wc{&st.abort_flag, args.status, args.timeout_ns};
  const int k_steps = (args.k_bytes + KB - 1) / KB;
  const int dm = nclusters / args.n_tiles, dn = nclusters - dm * args.n_tiles;
  TileWalk<TILE_M> walk;
  walk.start(cluster, args.n_tiles, args.groups, st.groups.mt_start);

  if (warp < 3) {
    // The issuing warps run their loops with all lanes and elect one to issue: with
    // one lane in the loop a K step took 960 cycles to issue, twice its MMAs' time.
    const uint32_t smem0 = smem_u32(smem), sfb0 = smem0 + S::kOffSfb;
    if (warp == 0 || warp == 2) {
      // ------------------------------------------------ TMA producers (both CTAs):
      // A and B's scales, and the barrier's byte count (warp 0); B (warp 2)
      int stage = 0;
      uint32_t phase = 0;
      uint32_t armed = 0, armed_parity = 0;
      bool ok = true;
      const uint32_t full0 = mapa_shared(smem_u32(&st.full[0]), 0);  // the leader's barriers
      for (int tile = cluster; ok && tile < total; tile += nclusters) {
        if (tile != cluster) walk.next(dm, dn, args.n_tiles, args.groups, st.groups.mt_start);
        const Tile t = walk.tile(st.groups.mt_start, st.groups.row_start);
        const int a_row = t.row0 + BM * (int)rank;
        const int b_row = (t.nt * args.n_out_tile + (int)rank * args.b_second) >> 2;
        const bool load_a = t.rows > BM * (int)rank;  // a half without rows loads none
        const int n0 = t.nt * args.n_out_tile, n1 = n0 + args.b_second;
        int sf_row = t.g * args.words;
        const uint32_t tx = 2 * (B_BYTES + 2 * S::kWords * SF_BYTES) + A_BYTES +
                            (t.rows > BM ? A_BYTES : 0);
        int kb = 0;
        for (int ks = 0; ks < k_steps; ++ks) {
          if (!__all_sync(FULL, mbar_wait(&st.empty[stage], phase ^ 1u, wc, 61))) {
            ok = false;
            break;
          }
          const uint32_t full = full0 + 8 * stage;
          const uint32_t sa = smem0 + stage * STAGE_BYTES;
          if (elect_one()) {
            if (warp == 0) {
              if (leader) mbar_arrive_expect_tx(&st.full[stage], tx);
              if (load_a) tma_load_2d_at(sa, &tmA, full, kb, a_row);
              const uint32_t sb = sfb0 + stage * S::kSfb;
              tma_load_2d_at(sb, &tmSB, full, n0, sf_row);
              tma_load_2d_at(sb + S::kWords * SF_BYTES, &tmSB, full, n1, sf_row);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tma_load_4d_at(sa + A_BYTES + j * B_BOX * KB, &tmB, full, kb, j, b_row, t.g);
            }
          }
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          kb += KB;
          sf_row += S::kWords;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) {  // both CTAs' loads are counted on the leader's barriers
        for (int s = 0; s < STAGES; ++s)
          if ((armed >> s) & 1u)
            mbar_wait_drain(&st.full[s], (armed_parity >> s) & 1u, args.timeout_ns);
      }
    } else if (warp == 1 && leader) {
      // ------------------------------------------------ B's scales to TMEM and pair MMAs (leader)
      constexpr int SFA_STEPS = SFA_WORDS / S::kWords;  // K steps per buffer of A's scales
      int stage = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0, sfa_phase = 0;
      bool ok = true;
      const uint64_t da0 = sdesc_kmajor_sw128(smem0), dsfb0 = sdesc_rows16(sfb0),
                     dsfa0 = sdesc_rows16(smem0 + S::kOffSfa);
      const int last = args.k_bytes - (k_steps - 1) * KB;  // bytes of a row in the last step
      for (int tile = cluster; ok && tile < total; tile += nclusters) {
        int chunk_left = 0;
        uint64_t dsfa = dsfa0;
        for (int ks = 0; ks < k_steps; ++ks) {
          if (chunk_left == 0) {
            if (!__all_sync(FULL, mbar_wait(&st.sfa_full[buf], sfa_phase, wc, 66))) {
              ok = false;
              break;
            }
            mbar_acquire_cluster(&st.sfa_full[buf], sfa_phase);  // the peer's words
            chunk_left = SFA_STEPS;
            dsfa = dsfa0 + static_cast<uint64_t>(buf * (SFA_BYTES >> 4));
          }
          if (!__all_sync(FULL, mbar_wait(&st.full[stage], phase, wc, 63))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          --chunk_left;
          const bool chunk_done = chunk_left == 0 || ks + 1 == k_steps;
          const uint32_t sfa = tmem_base + TMEM_SF + 32 * stage, sfb = sfa + TMEM_SFB;
          const uint64_t dsfb = dsfb0 + static_cast<uint64_t>(stage * (S::kSfb >> 4));
          const uint64_t da = da0 + static_cast<uint64_t>(stage * (STAGE_BYTES >> 4));
          const uint64_t db = da + (A_BYTES >> 4);
          if (elect_one()) {
#pragma unroll
            for (int w = 0; w < S::kWords; ++w) {
              tmem_copy_sf_pair(sfa + 4 * w, dsfa + w * (SF_BYTES >> 4));
#pragma unroll
              for (int hb = 0; hb < 2; ++hb)
                tmem_copy_sf_pair(sfb + 8 * w + 4 * hb,
                                  dsfb + (S::kWords * hb + w) * (SF_BYTES >> 4));
            }
          }
          // the accumulator is needed only now: with the scales and operands waited for
          // after it, the tensor cores idled 1,000 cycles more at every tile's start
          if (ks == 0 && !__all_sync(FULL, mbar_wait(&st.tempty, acc_phase ^ 1u, wc, 62))) {
            ok = false;
            break;
          }
          if (ks == 0) tc_fence_after_sync();
          if (elect_one()) {
            // 32 bytes of every row per MMA; the scale word, and the byte in it
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (ks + 1 < k_steps || kk * 32 < last)
                umma_mx_pair<FMT>(
                    tmem_base, da + 2 * kk, db + 2 * kk,
                    idesc_sf(idesc_mx<FMT>(TILE_M, BN), FMT == MOE_MXFP8 ? kk : 2 * (kk & 1)),
                    sfa + 4 * (kk * S::kWords / 4), sfb + 8 * (kk * S::kWords / 4),
                    (ks | kk) != 0 ? 1u : 0u);
            umma_commit_pair_mask(&st.empty[stage], 0x3);
            if (chunk_done) umma_commit_pair_mask(&st.sfa_empty[buf], 0x3);
            if (ks + 1 == k_steps) umma_commit_pair_mask(&st.tfull, 0x3);
          }
          dsfa += S::kWords * (SF_BYTES >> 4);
          if (chunk_done) {
            chunk_left = 0;
            buf ^= 1;
            if (buf == 0) sfa_phase ^= 1u;
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        acc_phase ^= 1u;
      }
      if (elect_one()) {
        umma_commit_pair_mask(&st.drain, 0x1);  // all of this warp's MMAs are done
        mbar_wait_drain(&st.drain, 0, args.timeout_ns);
      }
      __syncwarp();
    }
  } else if (warp == 3) {
    // ------------------------------------------------ scales of this CTA's rows of A
    const uint32_t full_leader[2] = {mapa_shared(smem_u32(&st.sfa_full[0]), 0),
                                     mapa_shared(smem_u32(&st.sfa_full[1]), 0)};
    const uint32_t sfa0 = smem_u32(smem) + S::kOffSfa + 16 * lane;
    int buf = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = cluster; ok && tile < total; tile += nclusters) {
      if (tile != cluster) walk.next(dm, dn, args.n_tiles, args.groups, st.groups.mt_start);
      const Tile t = walk.tile(st.groups.mt_start, st.groups.row_start);
      const int rows = min(BM, t.rows - BM * (int)rank);  // may be <= 0
      const uint32_t* src = args.a_scales + t.row0 + BM * (int)rank + lane;
      for (int w0 = 0; w0 < args.words; w0 += SFA_WORDS) {
        // words of rows lane + 32 j, 8 words at a time; the first are loaded while
        // the buffer is still in use
        const int nw = min(SFA_WORDS, args.words - w0);
        uint32_t v[8][4];
        auto load = [&](int h) {
#pragma unroll
          for (int w = 0; w < 8; ++w)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[w][j] = h + w < nw && lane + 32 * j < rows
                            ? src[(size_t)(w0 + h + w) * args.rows + 32 * j]
                            : 0u;
        };
        auto store = [&](int h) {
#pragma unroll
          for (int w = 0; w < 8; ++w)
            st_shared_v4(sfa0 + buf * SFA_BYTES + (h + w) * SF_BYTES, v[w]);
        };
        load(0);
        if (!__all_sync(FULL, mbar_wait(&st.sfa_empty[buf], phase ^ 1u, wc, 65))) {
          ok = false;
          break;
        }
        store(0);
        if (nw > 8) {
          load(8);
          store(8);
        }
        fence_proxy_async_smem();  // these writes -> tcgen05.cp
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(full_leader[buf]);
        buf ^= 1;
        if (buf == 0) phase ^= 1u;
      }
    }
  } else {
    // ------------------------------------------------ epilogue warps 4..19 (both CTAs)
    const int q = warp & 3;
    const int part = (warp - EPI_WARP0) >> 2;
    const int r_in_tile = q * 32 + lane;
    const uint32_t tempty_leader = mapa_shared(smem_u32(&st.tempty), 0);
    const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t out = smem_u32(smem) + S::kOffOut;
    uint32_t acc_phase = 0;
    for (int tile = cluster; tile < total; tile += nclusters) {
      if (tile != cluster) walk.next(dm, dn, args.n_tiles, args.groups, st.groups.mt_start);
      Tile t = walk.tile(st.groups.mt_start, st.groups.row_start);
      t.row0 += BM * (int)rank;
      t.rows = max(0, min(BM, t.rows - BM * (int)rank));
      const bool ok = __all_sync(FULL, mbar_wait(&st.tfull, acc_phase, wc, 64));
      if (!epilogue_agrees<EPI>(q, ok)) break;
      tc_fence_after_sync();
      uint32_t v[EPI_COLS];
      load_part<EPI>(tb, part, v);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(tempty_leader);
      store_part<FMT, EPI>(args, v, t, r_in_tile, part, out);
      acc_phase ^= 1u;
    }
    // the last tile's copies have left shared memory and are written
    if constexpr (EPI == MX_ROWS) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  // both CTAs are done with the accumulator and the scales before either frees TMEM or exits
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// Rows of codes in boxes of 128 bytes x 128 rows; bytes past a row's end and
// rows past the last one read 0.
cudaError_t make_tmap_a(CUtensorMap* map, const void* base, uint64_t rows, uint64_t row_bytes) {
  const cuuint64_t dims[2] = {row_bytes, rows}, strides[1] = {row_bytes};
  const cuuint32_t box[2] = {KB, BM};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box,
                CU_TENSOR_MAP_SWIZZLE_128B);
}

// The matrices' rows 4q + j in boxes of 128 bytes x one j x 32 q.
cudaError_t make_tmap_b(CUtensorMap* map, const void* base, uint64_t groups, uint64_t rows,
                        uint64_t row_bytes) {
  const cuuint64_t dims[4] = {row_bytes, 4, rows / 4, groups};
  const cuuint64_t strides[3] = {row_bytes, 4 * row_bytes, rows * row_bytes};
  const cuuint32_t box[4] = {KB, 1, B_BOX, 1};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box,
                CU_TENSOR_MAP_SWIZZLE_128B);
}

// The matrices' scale words, 128 columns of one K step a box.
cudaError_t make_tmap_sb(CUtensorMap* map, const void* base, uint64_t word_rows, uint64_t rows,
                         uint32_t step_words) {
  const cuuint64_t dims[2] = {rows, word_rows}, strides[1] = {rows * 4};
  const cuuint32_t box[2] = {BM, step_words};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, base, dims, strides, box,
                CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <int FMT, int EPI>
cudaError_t launch(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmSB,
                   const MxGemmArgs& args, int grid, cudaStream_t stream) {
  constexpr size_t smem = Shape<FMT, EPI>::kOffTail + sizeof(SmemTail);
  static_assert(smem <= 227 * 1024, "shared memory");
  static std::atomic<int> smem_set[MAX_DEVICES];
  const cudaError_t e =
      set_smem_limit_per_device(grouped_mx_kernel<FMT, EPI>, (int)smem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_chained(grouped_mx_kernel<FMT, EPI>, dim3(grid), dim3(THREADS), smem, stream, tmA,
                        tmB, tmSB, args);
}

// Rows of narrow tokens in expert order: codes[r] = tokens[tok_of[r]] and the
// words of scales; a token outside [0, T) gives zeros.  A block takes 32 rows, a
// warp four of them, whose 512-byte pieces are in flight together.  Bound by the
// writes: 155,296 rows of 2,048 bytes are 318 MB, 81 us at the 3.9 TB/s that
// writes alone reach here.
constexpr int GATHER_ROWS = 32;

__global__ void __launch_bounds__(256)
    gather_mx_kernel(const uint4* __restrict__ codes, const uint32_t* __restrict__ scales,
                     const int* __restrict__ tok_of, int T, int R, int vecs, int words,
                     uint4* __restrict__ codes_out, uint32_t* __restrict__ scales_out) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * GATHER_ROWS;
  const int rows = min(GATHER_ROWS, R - row0);
  int mine = lane < rows ? tok_of[row0 + lane] : -1;  // the token of row lane
  if (mine >= T) mine = -1;
  for (int c0 = 0; c0 < vecs; c0 += 32) {
    const int c = c0 + lane;
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = __shfl_sync(FULL, mine, warp * 4 + j);
      v[j] = t >= 0 && c < vecs ? codes[(size_t)t * vecs + c] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (warp * 4 + j < rows && c < vecs) codes_out[(size_t)(row0 + warp * 4 + j) * vecs + c] = v[j];
  }
  for (int w = warp; w < words; w += 8)
    if (lane < rows)
      scales_out[(size_t)w * R + row0 + lane] = mine >= 0 ? scales[(size_t)w * T + mine] : 0u;
}

}  // namespace

cudaError_t launch_grouped_mx(int fmt, int epi, const void* a, const void* b, MxGemmArgs args,
                              cudaStream_t stream) {
  if (args.groups > MX_MAX_GROUPS || args.tok_of) return cudaErrorInvalidValue;
  CUtensorMap tmA, tmB, tmSB;
  cudaError_t e;
  if ((e = make_tmap_a(&tmA, a, args.rows, args.k_bytes)) != cudaSuccess) return e;
  if ((e = make_tmap_b(&tmB, b, args.groups, args.n_rows, args.k_bytes)) != cudaSuccess) return e;
  if ((e = make_tmap_sb(&tmSB, args.b_scales, (uint64_t)args.groups * args.words, args.n_rows,
                        fmt == MOE_MXFP8 ? 1 : 2)) != cudaSuccess)
    return e;
  args.n_out_tile = epi == MX_SWIGLU ? BN / 2 : BN;
  args.n_tiles = (args.n_valid + args.n_out_tile - 1) / args.n_out_tile;
  args.b_second = epi == MX_SWIGLU ? args.n_valid : BN / 2;
  const long long tiles = ((long long)args.rows / TILE_M + args.groups) * args.n_tiles;
  const int sms = num_sms() & ~1;
  const int grid = (int)(2 * tiles < sms ? 2 * tiles : sms);
  if (fmt == MOE_MXFP8)
    return epi == MX_SWIGLU ? launch<MOE_MXFP8, MX_SWIGLU>(tmA, tmB, tmSB, args, grid, stream)
                            : launch<MOE_MXFP8, MX_ROWS>(tmA, tmB, tmSB, args, grid, stream);
  return epi == MX_SWIGLU ? launch<MOE_MXFP4, MX_SWIGLU>(tmA, tmB, tmSB, args, grid, stream)
                          : launch<MOE_MXFP4, MX_ROWS>(tmA, tmB, tmSB, args, grid, stream);
}

cudaError_t launch_gather_mx(const uint8_t* codes, const uint8_t* scales, const int* tok_of, int T,
                             int R, int row_bytes, int words, uint8_t* codes_out,
                             uint8_t* scales_out, cudaStream_t stream) {
  const int vecs = row_bytes / 16;
  const unsigned blocks = (R + GATHER_ROWS - 1) / GATHER_ROWS;
  return launch_chained(gather_mx_kernel, dim3(blocks), dim3(256), 0, stream,
                        reinterpret_cast<const uint4*>(codes),
                        reinterpret_cast<const uint32_t*>(scales), tok_of, T, R, vecs, words,
                        reinterpret_cast<uint4*>(codes_out),
                        reinterpret_cast<uint32_t*>(scales_out));
}

}  // namespace rmoe
