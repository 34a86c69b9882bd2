// Grouped products of MX operands for few rows per group: the product of
// grouped_mx.cu with its operands swapped, D^T = W . X^T.
//
// With 15 rows an expert a 256-row tile spends its MMA time on padding and its
// tile's fixed costs on little work, and the weights' stream, which bounds such
// a call, waits for both.  Here 128 weight rows fill the MMA's M and at most C = 64,
// 96 or 128 rows of a group its N (a multiple of 16), so that an MMA takes a quarter
// to half of the time; one CTA per SM works alone, with 80 to 128 KB of weights in
// flight and two accumulators.
//
// Work item = (chunk of at most C rows of one group, 128 weight rows):
//   MX_ROWS    out[dest(r), n0 + l] = bf16( row_w[r] * D[l, r] )
//   MX_SWIGLU  gate rows i0.. and up rows I + i0.. of the weights in two
//              accumulators: lane l has gate and up of output column i0 + l; the
//              32 lanes of a warp are one block of h, its largest element by a
//              warp reduction.
// Scales: both operands' words come by plain loads into the order that
// tcgen05.cp wants (mx_mma.cuh), 8 words a row at a time, two buffers.
// Warp roles: warp 0 TMA loads; warp 1 TMEM, scales to TMEM, MMAs; warp 2 the
// weights' scales (of the gate rows), warp 3 those of the up rows and of the
// rows; warps 4..11 the epilogue.  Every wait but that for tensor memory is bounded
// (common.cuh).
//
// HBM bounds it: 1,920 rows of 128 groups, K = 1024, N = 1536, MXFP8: 36.0 us for 216
// MB (6.0 TB/s, 0.93 of the measured copy; pair tiles 51 us); 6,272 rows, K = 768, N =
// 2048: MXFP8 39.7 us for 238 MB (6.0 TB/s; pair tiles 53.7), MXFP4 28.0 for 135 MB
// (4.8 TB/s; 38.7).  One row: the latency of a K step after the other, 8 rows of 8
// groups, K = 8192, MXFP8: 14.7 us, 220 ns a stage.  That issue time was the bound
// throughout before: with shared memory aligned at run time (addresses then live in
// ordinary registers, and every barrier and descriptor costs more instructions) and one
// K step a stage, 25 us, and the calls above 38.5, 43.0 and 29.8.
//
// Shared memory: rows of bf16 177 KB (items of 64 rows, three stages), 225 KB (four) and
// 209 KB (items of 128 rows), SwiGLU 185 KB (64 rows) and 201 KB (96 rows).  Every form
// leaves room on its SM (228 KB, of which each block takes 1 KB more than its own) for
// a block without shared memory, as those of the next call's gathering copy are, which
// starts early: with less the experts of 64 tokens took 108 us instead of 103, because
// the copy had to wait for this kernel.
#include "mx_mma.cuh"

namespace rmoe {

namespace {

constexpr int WM = 128;           // weight rows per item (the MMA's M)
constexpr int KB = 128;           // bytes of a row per K step
constexpr int XBOX = 32;          // rows per TMA box
constexpr int W_BYTES = WM * KB;
constexpr int OUT_PITCH = 2 * WM; // bytes of an output row in shared memory
constexpr int THREADS = 384;
constexpr int EPI_WARP0 = 4;
constexpr int EPI_WARPS = 8;      // two for each 32 columns, 16 rows in turn
constexpr int SF_WORDS = 8;       // words per row in a buffer of scales
constexpr int MAX_STAGES = 5;
constexpr uint32_t TMEM_COLS = 512;

// C: rows per item at most (the MMA's N, padded to 16).
template <int FMT, int EPI, int C, int STAGES>
struct Shape {
  static constexpr int kWords = FMT == MOE_MXFP8 ? 1 : 2;  // scale words per row and K step
  static constexpr int kTiles = EPI == MX_SWIGLU ? 2 : 1;  // weight tiles per item
  static constexpr int kXBytes = C * KB;
  static constexpr int kStepBytes = kTiles * W_BYTES + kXBytes;
  static constexpr int kSub = C == 64 ? 2 : 1;  // K steps per stage
  static constexpr int kStageBytes = kSub * kStepBytes;
  static constexpr int kStages = STAGES;
  static constexpr uint32_t kAcc = kTiles * C;   // TMEM columns of an accumulator (gate, up)
  static constexpr uint32_t kTmemSf = 2 * kAcc;  // + 32 per step: 4 per word of each tile, rows first
  static constexpr int kSfBytes = SF_WORDS * MX_SF_BYTES;  // per operand tile and buffer
  static constexpr int kSfBuf = (kTiles + 1) * kSfBytes;   // the rows', then the weights'
  static constexpr int kOffSf = kStages * kStageBytes;
  static constexpr int kOffOut = kOffSf + 2 * kSfBuf;
  static constexpr int kOffTail = kOffOut + (EPI == MX_ROWS ? C * OUT_PITCH : 0);
  static_assert(kStages <= MAX_STAGES && kTmemSf + 32 * kSub * kStages <= TMEM_COLS, "TMEM");
};

struct __align__(8) SmemTail {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t sf_full[2];
  uint64_t sf_empty[2];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  MxGroups groups;
};

template <int FMT>
__device__ __forceinline__ void umma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (FMT == MOE_MXFP8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_copy_sf(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
               : "memory");
}

// The same of the rows in `at` (lane l: those of rows l, l + 32, ..; -1: zeros).
template <int J>
__device__ __forceinline__ void load_words_at(uint32_t (&v)[SF_WORDS][4], const uint32_t* src,
                                              size_t pitch, int nw, const int (&at)[J]) {
#pragma unroll
  for (int w = 0; w < SF_WORDS; ++w)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[w][j] = j < J && w < nw && at[j] >= 0 ? src[w * pitch + at[j]] : 0u;
}

// The tokens of an item's rows (lane l: rows l, l + 32, ..); -1: none, or outside [0, T).
template <int J>
__device__ __forceinline__ void item_tokens(const MxGemmArgs& a, const Tile& t, int lane,
                                            int (&tok)[J]) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int n = lane + 32 * j;
    tok[j] = n < t.rows ? a.tok_of[t.row0 + n] : -1;
    if (tok[j] >= a.a_rows) tok[j] = -1;
  }
}

// Scale words [w0, w0 + nw) of `rows` rows (`src` + lane + 32 j of each word, `pitch`
// words from one word to the next) into a buffer: 16-byte row l of a word holds
// those of rows l, l + 32, l + 64, l + 96.
template <int J>
__device__ __forceinline__ void load_words(uint32_t (&v)[SF_WORDS][4], const uint32_t* src,
                                           size_t pitch, int nw, int rows, int lane) {
#pragma unroll
  for (int w = 0; w < SF_WORDS; ++w)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[w][j] = j < J && w < nw && lane + 32 * j < rows ? src[w * pitch + lane + 32 * j] : 0u;
}

__device__ __forceinline__ void store_words(uint32_t addr, const uint32_t (&v)[SF_WORDS][4]) {
#pragma unroll
  for (int w = 0; w < SF_WORDS; ++w) st_shared_v4(addr + w * MX_SF_BYTES, v[w]);
}

__device__ __forceinline__ void st_shared_b16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// v[n / 32], n the same in all lanes.
template <typename V, int J>
__device__ __forceinline__ V of_row(const V (&v)[J], int n) {
  V r = v[0];
#pragma unroll
  for (int j = 1; j < J; ++j) r = n >= 32 * j ? v[j] : r;
  return r;
}

// GATHER: row r of the groups is row tok_of[r] of X, loaded by a TMA box of its own.
template <int FMT, int EPI, int C, int STAGES, bool GATHER>
__global__ void __launch_bounds__(THREADS, 1)
    grouped_mx_few_kernel(const __grid_constant__ CUtensorMap tmW,
                          const __grid_constant__ CUtensorMap tmX, const MxGemmArgs args) {
  using S = Shape<FMT, EPI, C, STAGES>;
  constexpr int SUB = S::kSub;
  extern __shared__ __align__(1024) uint8_t smem[];
  SmemTail& st = *reinterpret_cast<SmemTail*>(smem + S::kOffTail);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&st.full[s], 1);
      mbar_init(&st.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&st.sf_full[b], 2);
      mbar_init(&st.sf_empty[b], 1);
      mbar_init(&st.tfull[b], 1);
      mbar_init(&st.tempty[b], EPI_WARPS);
    }
    mbar_init(&st.drain, 1);
    st.abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  // What comes before reads nothing that an earlier kernel writes.  After the up
  // product (args.after_up) only its rows have to be waited for: it lets this
  // kernel start when all that came before it was complete, so the group table
  // and the weights can be read while it runs.
  const bool early = EPI == MX_ROWS && args.after_up != 0;
  if (!early) pdl_wait();
  const int total = mx_group_table<C>(args, st.groups) * args.n_tiles;
  const WaitCtx wc{&st.abort_flag, args.status, args.timeout_ns};
  const int first = blockIdx.x, step = gridDim.x;
  uint32_t tmem_base = 0;  // warp 1 and the epilogue
  if (first < total) {
    const int k_steps = (args.k_bytes + KB - 1) / KB;
    const int* mts = st.groups.mt_start;
    const int* rs = st.groups.row_start;
    const int dm = step / args.n_tiles, dn = step - dm * args.n_tiles;
    TileWalk<C> walk;
    walk.start(first, args.n_tiles, args.groups, mts);
    const uint32_t smem0 = smem_u32(smem), sf0 = smem0 + S::kOffSf;

    if (warp == 0) {
      // ------------------------------------------------ TMA producer
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_parity = 0;
      bool ok = true;
      int ahead = 0;  // steps of the first item whose weights are loaded before the rows
      for (int item = first; ok && item < total; item += step) {
        if (item != first) walk.next(dm, dn, args.n_tiles, args.groups, mts);
        const Tile t = walk.tile(mts, rs);
        const int w_row = t.nt * WM;
        const int nb = (t.rows + XBOX - 1) / XBOX;
        const uint32_t tx = S::kTiles * W_BYTES + (GATHER ? t.rows : nb * XBOX) * KB;
        int tok[C / 32];
        if constexpr (GATHER) item_tokens(args, t, lane, tok);
        auto load_weights = [&](int st_i, int ks) {  // one lane
          uint8_t* sw = smem + (size_t)st_i * S::kStageBytes + S::kXBytes;
          const int n = min(SUB, k_steps - ks);
          mbar_arrive_expect_tx(&st.full[st_i], n * tx);
#pragma unroll
          for (int u = 0; u < SUB; ++u)
            if (u < n)
#pragma unroll
              for (int w = 0; w < S::kTiles; ++w)
                tma_load_3d(sw + u * S::kStepBytes + w * W_BYTES, &tmW, &st.full[st_i],
                            (ks + u) * KB, w_row + w * args.b_second, t.g);
        };
        if (early && item == first) {
          ahead = min(S::kStages, (k_steps + SUB - 1) / SUB);
          if (elect_one())
            for (int s = 0; s < ahead; ++s) load_weights(s, s * SUB);
          __syncwarp();
          pdl_wait();
        }
        for (int ks = 0; ks < k_steps; ks += SUB) {
          if (!__all_sync(FULL, mbar_wait(&st.empty[stage], phase ^ 1u, wc, 71))) {
            ok = false;
            break;
          }
          uint8_t* sx = smem + (size_t)stage * S::kStageBytes;
          const int steps = min(SUB, k_steps - ks);
          if (elect_one()) {
            if (ahead == 0) load_weights(stage, ks);
            if constexpr (!GATHER)
              for (int u = 0; u < steps; ++u)
                for (int b = 0; b < nb; ++b)
                  tma_load_2d(sx + u * S::kStepBytes + b * XBOX * KB, &tmX, &st.full[stage],
                              (ks + u) * KB, t.row0 + b * XBOX);
          }
          if (ahead > 0) --ahead;
          if constexpr (GATHER) {
            const bool lead = elect_one();
            for (int n = 0; n < t.rows; ++n) {
              const int r = __shfl_sync(FULL, of_row(tok, n), n & 31);
              // a row past the last one reads zeros
              if (lead)
                for (int u = 0; u < steps; ++u)
                  tma_load_2d(sx + u * S::kStepBytes + n * KB, &tmX, &st.full[stage],
                              (ks + u) * KB, r < 0 ? args.a_rows : r);
            }
          }
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        for (int s = 0; s < S::kStages; ++s)
          if ((armed >> s) & 1u)
            mbar_wait_drain(&st.full[s], (armed_parity >> s) & 1u, args.timeout_ns);
      }
    } else if (warp == 1) {
      // ------------------------------------------------ scales to TMEM and MMAs
      // All of TMEM, which has no wait with a limit: behind the wait for the kernels
      // before, one of which could otherwise be waiting for it, and before the kernel
      // after may start, which could otherwise take it first and wait for this one.
      // The first operands are on their way meanwhile.
      if (early) pdl_wait();
      tmem_alloc(&st.tmem_base, TMEM_COLS);
      tmem_relinquish();
      tc_fence_before_sync();
      warps_sync<1 + EPI_WARPS>(2);
      tc_fence_after_sync();
      tmem_base = uniform(st.tmem_base);
      // (also not before the wait because the kernel after may be an early one)
      pdl_launch_dependents();
      constexpr int SF_STEPS = SF_WORDS / S::kWords;  // K steps per buffer of scales
      int stage = 0, buf = 0, acc = 0;
      uint32_t phase = 0, sf_phase = 0, acc_phase = 0;
      bool ok = true;
      const uint64_t dx0 = sdesc_kmajor_sw128(smem0), dsf0 = sdesc_rows16(sf0);
      for (int item = first; ok && item < total; item += step) {
        if (item != first) walk.next(dm, dn, args.n_tiles, args.groups, mts);
        const Tile t = walk.tile(mts, rs);
        const uint32_t idesc = idesc_mx<FMT>(WM, (t.rows + 15) & ~15);
        const uint32_t d = tmem_base + acc * S::kAcc;
        int chunk_left = 0;
        uint64_t dsf = dsf0;
        for (int ks = 0; ks < k_steps; ks += SUB) {
          if (chunk_left == 0) {
            if (!__all_sync(FULL, mbar_wait(&st.sf_full[buf], sf_phase, wc, 72))) {
              ok = false;
              break;
            }
            chunk_left = SF_STEPS;
            dsf = dsf0 + static_cast<uint64_t>(buf * (S::kSfBuf >> 4));
          }
          if (!__all_sync(FULL, mbar_wait(&st.full[stage], phase, wc, 73))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          chunk_left -= SUB;
          const bool chunk_done = chunk_left == 0 || ks + SUB >= k_steps;
          const uint32_t sf0 = tmem_base + S::kTmemSf + 32 * SUB * stage;
          const uint64_t dx0s = dx0 + static_cast<uint64_t>(stage * (S::kStageBytes >> 4));
          if (elect_one()) {
#pragma unroll
            for (int u = 0; u < SUB; ++u)  // (past the last step: words that nothing uses)
#pragma unroll
              for (int o = 0; o < S::kTiles + 1; ++o)
#pragma unroll
                for (int w = 0; w < S::kWords; ++w)
                  tmem_copy_sf(sf0 + 32 * u + 4 * (S::kWords * o + w),
                               dsf + ((o * S::kSfBytes + (u * S::kWords + w) * MX_SF_BYTES) >> 4));
          }
          if (ks == 0) {
            if (!__all_sync(FULL, mbar_wait(&st.tempty[acc], acc_phase ^ 1u, wc, 74))) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
          }
          if (elect_one()) {
            // 32 bytes of every row per MMA; the scale word, and the byte in it
            auto mma = [&](int u, int kk) {
              const uint64_t dx = dx0s + u * (S::kStepBytes >> 4);
              const uint32_t sf = sf0 + 32 * u, word = 4 * (kk * S::kWords / 4);
              const uint32_t id = idesc_sf(idesc, FMT == MOE_MXFP8 ? kk : 2 * (kk & 1));
#pragma unroll
              for (int w = 0; w < S::kTiles; ++w)
                umma_mx<FMT>(d + w * C, dx + ((S::kXBytes + w * W_BYTES) >> 4) + 2 * kk,
                             dx + 2 * kk, id, sf + 4 * S::kWords * (1 + w) + word, sf + word,
                             (ks | u | kk) != 0 ? 1u : 0u);
            };
            if (ks + SUB < k_steps) {
#pragma unroll
              for (int m = 0; m < 4 * SUB; ++m) mma(m >> 2, m & 3);
            } else {
#pragma unroll
              for (int m = 0; m < 4 * SUB; ++m)
                if (ks * KB + m * 32 < args.k_bytes) mma(m >> 2, m & 3);
            }
            umma_commit(&st.empty[stage]);
            if (chunk_done) umma_commit(&st.sf_empty[buf]);
            if (ks + SUB >= k_steps) umma_commit(&st.tfull[acc]);
          }
          dsf += SUB * S::kWords * (MX_SF_BYTES >> 4);
          if (chunk_done) {
            chunk_left = 0;
            buf ^= 1;
            if (buf == 0) sf_phase ^= 1u;
          }
          if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (elect_one()) {
        umma_commit(&st.drain);  // all of this warp's MMAs are done
        mbar_wait_drain(&st.drain, 0, args.timeout_ns);
      }
      __syncwarp();
    } else if (warp < EPI_WARP0) {
      // ------------------------------------------------ scales (warp 2: weight tile 0; 3: the rest)
      if (early && warp == 3) pdl_wait();
      int buf = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int item = first; ok && item < total; item += step) {
        if (item != first) walk.next(dm, dn, args.n_tiles, args.groups, mts);
        const Tile t = walk.tile(mts, rs);
        int tok[C / 32];
        if constexpr (GATHER)
          if (warp == 3) item_tokens(args, t, lane, tok);
        for (int w0 = 0; w0 < args.words; w0 += SF_WORDS) {
          const int nw = min(SF_WORDS, args.words - w0);
          const int n0 = t.nt * WM + (warp == 2 ? 0 : args.b_second);  // first weight row
          const uint32_t* wsrc =
              args.b_scales + ((size_t)t.g * args.words + w0) * args.n_rows + n0;
          const uint32_t dst = sf0 + buf * S::kSfBuf + 16 * lane;
          uint32_t v[SF_WORDS][4], x[SF_WORDS][4];
          if (warp == 2 || S::kTiles == 2)
            load_words<4>(v, wsrc, args.n_rows, nw, args.n_rows - n0, lane);
          if (warp == 3) {
            const uint32_t* xsrc = args.a_scales + (size_t)w0 * args.a_rows;
            if constexpr (GATHER)
              load_words_at(x, xsrc, args.a_rows, nw, tok);
            else
              load_words<C / 32>(x, xsrc + t.row0, args.a_rows, nw, t.rows, lane);
          }
          if (!__all_sync(FULL, mbar_wait(&st.sf_empty[buf], phase ^ 1u, wc, 75))) {
            ok = false;
            break;
          }
          if (warp == 2 || S::kTiles == 2)
            store_words(dst + (warp == 2 ? 1 : 2) * S::kSfBytes, v);
          if (warp == 3) store_words(dst, x);
          fence_proxy_async_smem();  // these writes -> tcgen05.cp
          __syncwarp();
          if (lane == 0) mbar_arrive(&st.sf_full[buf]);
          buf ^= 1;
          if (buf == 0) phase ^= 1u;
        }
      }
    } else {
      // ------------------------------------------------ epilogue warps 4..11
      if (early) pdl_wait();
      warps_sync<1 + EPI_WARPS>(2);
      tc_fence_after_sync();
      tmem_base = uniform(st.tmem_base);
      const int q = warp & 3, part = (warp - EPI_WARP0) >> 2;
      constexpr int COPIES = C / EPI_WARPS;  // MX_ROWS: rows that a warp copies, one a lane
      const uint32_t out = smem0 + S::kOffOut;
      int acc = 0;
      uint32_t acc_phase = 0;
      for (int item = first; item < total; item += step) {
        if (item != first) walk.next(dm, dn, args.n_tiles, args.groups, mts);
        const Tile t = walk.tile(mts, rs);
        const int col0 = t.nt * WM + q * 32;  // the warp's first output column
        const int crow = (warp - EPI_WARP0) * COPIES + lane;   // MX_ROWS: this lane's row of the copies,
        int dest = -1;                        // its output row (-1: none),
        float w[C / 32];                      // and the weights of rows l, l + 32, ..
        if constexpr (EPI == MX_ROWS) {
          if (lane < COPIES && crow < t.rows) {
            dest = args.row_dest ? args.row_dest[t.row0 + crow] : t.row0 + crow;
            if (dest >= args.out_rows) dest = -1;
          }
#pragma unroll
          for (int j = 0; j < C / 32; ++j) {
            const int n = lane + 32 * j;
            w[j] = args.row_w && n < t.rows ? args.row_w[t.row0 + n] : 1.0f;
          }
        }
        bool ok = __all_sync(FULL, mbar_wait(&st.tfull[acc], acc_phase, wc, 76));
        if constexpr (EPI == MX_ROWS) {
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the last item's copies
          ok = warps_agree<EPI_WARPS>(1, ok);
        }
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t tb =
            tmem_base + acc * S::kAcc + (static_cast<uint32_t>(q * 32) << 16);
        // 16 rows at a time, without branches between them: their shuffles,
        // reductions and stores overlap (row by row they cost 170 cycles each,
        // and bounded the call from 8 rows a group on)
#pragma unroll 1
        for (int n0 = 16 * part; n0 < t.rows; n0 += 32) {
          uint32_t g[16];
          tmem_ld_32x32b_x16(tb + n0, g);
          if constexpr (EPI == MX_ROWS) {
            // The rows go to shared memory and from there, 128 columns of a row at a
            // time, by bulk copies: stored from registers, 32 columns at a time, they
            // bounded the call (768 x 2048, 49 rows a group, MXFP4, items of 64 rows: 58.7
            // us, now 32.1; 15 rows 30.5, now 25.4).  Eight warps: four took 33.4, and
            // 36.4 instead of 29.8 with items of 128 rows.
            tmem_ld_wait();
            const uint32_t dst = out + n0 * OUT_PITCH + 2 * (q * 32 + lane);
            const float wl = of_row(w, n0);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float wj = __shfl_sync(FULL, wl, (n0 & 16) + j);
              st_shared_b16(dst + j * OUT_PITCH,
                            __bfloat16_as_ushort(__float2bfloat16_rn(wj * __uint_as_float(g[j]))));
            }
          } else {
            uint32_t u[16];
            tmem_ld_32x32b_x16(tb + C + n0, u);
            tmem_ld_wait();
            const int left = col0 < args.n_valid ? t.rows - n0 : 0;  // whole blocks of 32 columns
            const int row = t.row0 + n0;
            uint32_t bytes = 0;  // lane j: scale byte of row j
            float h[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              h[j] = silu_f(__uint_as_float(g[j])) * __uint_as_float(u[j]);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint32_t byte = mx_scale_byte<FMT>(
                  __reduce_max_sync(FULL, __float_as_uint(h[j]) & 0x7fffffffu));
              if (lane == j) bytes = byte;
              h[j] = byte == 255u ? 0.0f : h[j] * mx_inverse_scale(byte);
            }
            uint8_t* dst = static_cast<uint8_t*>(args.out) +
                           ((size_t)row * args.n_valid + col0) / MxFmt<FMT>::kPerByte;
            const int pitch = args.n_valid / MxFmt<FMT>::kPerByte;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if constexpr (FMT == MOE_MXFP8) {
                const uint8_t c = static_cast<uint8_t>(mx_pack_e4m3(h[j], 0.f, 0.f, 0.f));
                if (j < left) dst[(size_t)j * pitch + lane] = c;
              } else {
                const float o = __shfl_xor_sync(FULL, h[j], 1);
                const uint8_t c = mx_pack_e2m1_pair(h[j], o);
                if (j < left && (lane & 1) == 0) dst[(size_t)j * pitch + (lane >> 1)] = c;
              }
            }
            // a word's bytes past the last column's block are 0
            if (lane < t.rows - n0 && lane < 16)
              reinterpret_cast<uint8_t*>(args.out_scales + (size_t)t.nt * args.rows + row + lane)[q] =
                  static_cast<uint8_t>(left > 0 ? bytes : 0u);
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&st.tempty[acc]);
        if constexpr (EPI == MX_ROWS) {
          fence_proxy_async_smem();  // these writes -> the copies
          warps_sync<EPI_WARPS>(1);
          if (dest >= 0)
            bulk_store(static_cast<__nv_bfloat16*>(args.out) + (size_t)dest * args.n_valid +
                           t.nt * WM,
                       out + crow * OUT_PITCH, 2 * min(WM, args.n_valid - t.nt * WM));
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      // the last item's copies have left shared memory and are written
      if constexpr (EPI == MX_ROWS) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
  }

  // no CTA ends before the kernels that came before have: what follows this kernel
  // relies on that
  pdl_wait();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1 && first < total) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// Rows of codes in boxes of 128 bytes x box_rows; zeros past the ends.
cudaError_t make_tmap_rows(CUtensorMap* map, const void* base, uint64_t rows, uint64_t row_bytes,
                           uint32_t box_rows) {
  const cuuint64_t dims[2] = {row_bytes, rows}, strides[1] = {row_bytes};
  const cuuint32_t box[2] = {KB, box_rows};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t make_tmap_matrices(CUtensorMap* map, const void* base, uint64_t groups, uint64_t rows,
                               uint64_t row_bytes) {
  const cuuint64_t dims[3] = {row_bytes, rows, groups};
  const cuuint64_t strides[2] = {row_bytes, rows * row_bytes};
  const cuuint32_t box[3] = {KB, WM, 1};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int FMT, int EPI, int C, int STAGES, bool GATHER = false>
cudaError_t launch(const CUtensorMap& tmW, const CUtensorMap& tmX, const MxGemmArgs& args,
                   cudaStream_t stream) {
  constexpr size_t smem = Shape<FMT, EPI, C, STAGES>::kOffTail + sizeof(SmemTail);
  static_assert(smem + 2 * 1024 <= 228 * 1024, "shared memory: a small kernel's block beside it");
  static std::atomic<int> smem_set[MAX_DEVICES];
  auto kernel = grouped_mx_few_kernel<FMT, EPI, C, STAGES, GATHER>;
  const cudaError_t e = set_smem_limit_per_device(kernel, (int)smem, smem_set);
  if (e != cudaSuccess) return e;
  const long long items = ((long long)args.rows / C + args.groups) * args.n_tiles;
  const int sms = num_sms();
  return launch_chained(kernel, dim3((unsigned)(items < sms ? items : sms)), dim3(THREADS), smem,
                        stream, tmW, tmX, args);
}

// MX_ROWS: rows per group, on average, from which items hold up to 128 rows and not
// 64 (groups are uneven: fewer read their weights twice).  128 experts, K = 768, N =
// 2048, 64 / 128 rows an item: MXFP8 15 rows a group 38.0 / 38.8 us, 32 rows 41.5 /
// 40.2, 49 rows 48.9 / 43.0; MXFP4 25.4 / 25.4, 27.5 / 27.2, 32.1 / 29.8.  MX_SWIGLU,
// whose two accumulators leave room for 96: H = 2048, I = 768 with the down product
// after it, 49 rows 120.8 / 120.3 MXFP8 and 74.5 / 74.7 MXFP4, 96 rows 145 / 137 and
// 95.2 / 90.4.
constexpr long long WIDE_UP_ROWS = 64;
constexpr long long WIDE_ROWS = 24;

// Bytes of a row above which items of 64 rows get a fourth stage: MXFP8 K = 2048, N =
// 1536, 15 rows a group 66.6 us, with three 69.2; K = 768, N = 2048 36.0, with three 35.2;
// 1,024 bytes the same.
constexpr int DEEP_BYTES = 1024;

template <int FMT>
cudaError_t launch_fmt(const CUtensorMap& tmW, const CUtensorMap& tmX, const MxGemmArgs& args,
                       int epi, cudaStream_t stream) {
  if (args.tok_of)
    return epi == MX_SWIGLU ? launch<FMT, MX_SWIGLU, 64, 2, true>(tmW, tmX, args, stream)
                            : cudaErrorInvalidValue;
  if (epi == MX_SWIGLU)
    return args.rows > WIDE_UP_ROWS * args.groups
               ? launch<FMT, MX_SWIGLU, 96, 4>(tmW, tmX, args, stream)
               : launch<FMT, MX_SWIGLU, 64, 2>(tmW, tmX, args, stream);
  if (args.rows > WIDE_ROWS * args.groups)
    return launch<FMT, MX_ROWS, 128, 5>(tmW, tmX, args, stream);
  return args.k_bytes > DEEP_BYTES ? launch<FMT, MX_ROWS, 64, 4>(tmW, tmX, args, stream)
                                   : launch<FMT, MX_ROWS, 64, 3>(tmW, tmX, args, stream);
}

}  // namespace

cudaError_t launch_grouped_mx_few(int fmt, int epi, const void* a, const void* b, MxGemmArgs args,
                                  cudaStream_t stream) {
  if (args.groups > MX_MAX_GROUPS) return cudaErrorInvalidValue;
  CUtensorMap tmW, tmX;
  cudaError_t e;
  if ((e = make_tmap_matrices(&tmW, b, args.groups, args.n_rows, args.k_bytes)) != cudaSuccess)
    return e;
  if ((e = make_tmap_rows(&tmX, a, args.a_rows, args.k_bytes, args.tok_of ? 1 : XBOX)) !=
      cudaSuccess)
    return e;
  args.n_out_tile = WM;
  args.n_tiles = (args.n_valid + WM - 1) / WM;
  args.b_second = args.n_valid;  // MX_SWIGLU: the up rows
  return fmt == MOE_MXFP8 ? launch_fmt<MOE_MXFP8>(tmW, tmX, args, epi, stream)
                          : launch_fmt<MOE_MXFP4>(tmW, tmX, args, epi, stream);
}

}  // namespace rmoe
