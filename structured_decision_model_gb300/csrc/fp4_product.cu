// Products of microscaled 4-bit matrices on the 5th-generation tensor cores
// (tcgen05.mma kind::mxf4nvf4, block-scaled): y = x w^T with fp32 sums in TMEM, the blocks'
// scales applied by the tensor cores, the rows' scales, the bias and the LayerNorm fold in
// the epilogue.
//
// w's rows are the MMA's M side (TMEM lanes) and x's rows its N side (columns): a thread of
// the epilogue then holds one column of the output, with its scale, bias and sum in
// registers, and a warp stores 32 neighbouring values of an output row, whatever the
// output's width, stride and alignment are.
//
// A K tile is 256 columns: 128 bytes of codes a row (one 128-byte swizzle atom, four MMAs of
// 64 columns) and 2 (mxfp4) or 4 (nvfp4) 512-byte groups of scales for every 128 rows,
// which tcgen05.cp spreads over 4 TMEM columns each.  The tensor cores take the copies and
// the products of one thread in order, so one set of scale columns serves every K tile.
//
// Every wait is bounded: on a timeout the CTA sets the timeout flag, waits (bounded) for its
// own copies and MMAs in flight, frees TMEM and returns.
#include "fp4_tile.cuh"

namespace clef {

namespace {

// ------------------------------------------- CTA pairs, 256 x 256 tiles, persistent
// Many rows: two CTAs (cta_group::2) compute 256 rows of w x 256 rows of x, each loading its
// own 128 rows of w and half of x's rows (scales: of its rows of w, and of all rows of x), and
// walk the tiles until none is left.  Two 256-column accumulators and the scales do not fit
// 512 TMEM columns, so the accumulators share 64: [0, 256) and [192, 448), scales from 448 on.
// The epilogue takes the shared columns first and hands them back at once; from then on the next
// tile's products run beside the rest of it.
//
// What bounds it is power, and the MMAs themselves.  Sustained, a K tile takes 613 cycles at 1.62 GHz (nvfp4, K = 16384; mxfp4 597
// at 1.71), of which its four MMAs are 512; without loads and outputs 595 at 1.96 (578 at 2.07).  Loads cost clock,
// not cycles: 96.9 us with them, 78.8 without; without outputs 91.4, without copies of scales 96.1 (4864 x 4096 x 16384).
// An MMA's scales are copied before the MMA that comes before it: the copies
// run beside that one (all of a K tile's copies before its first MMA left the tensor cores idle: 650 and 609 us instead
// of 618 and 575; a K tile's last MMA held back behind the next one's first copies: 630 and 588).  131072 x 4096 x 4096
// to bf16 takes 614 to 625 us (7.1 PFLOP/s; mxfp4 578, 7.6), 4864 x 4096 x 16384 89 to 97 us (mxfp4 85 to 89).  One MMA
// thread in a diverged warp took 1527 us, a second election a K tile or a slower producer 715, hand-over by a releasing
// arrival (which waits for the last tile's stores) 10 % more; a last round in halves of tiles gained nothing.
// Outputs of fp32, or of rows that do not start or end on 16 bytes, go out by direct stores (emit).
template <int FMT>
struct PairCfg {
    static constexpr int GROUPS = groups_of(FMT);
    static constexpr int ROWS = 256;                          // rows of x in a tile
    static constexpr int X_BYTES = ROWS / 2 * kAtomBytes;     // a CTA's half
    static constexpr int S_BYTES = GROUPS * kFp4ScaleGroup;
    static constexpr int STAGE = kWBytes + X_BYTES + 3 * S_BYTES;
    static constexpr int STAGE_STRIDE = (STAGE + 1023) / 1024 * 1024;
    static constexpr int STAGES = 5;
    static constexpr int OUT_BYTES = 16 * kWRows * 2;         // a staged piece of the output: 16 rows x 128 columns
    static constexpr int SMEM = STAGES * STAGE_STRIDE + 4 * OUT_BYTES + 1024 + 2 * ROWS * 8 + 256;
    static constexpr uint32_t ACC1 = 192, S_AT = 448;
    static_assert(4 * GROUPS + 8 * GROUPS <= 64, "scales fit the last columns");
};

// BULK: 16-bit outputs whose rows start and end on 16 bytes, staged in shared memory and stored by TMA.
template <int FMT, int OUT, bool BULK>
__global__ void __launch_bounds__(kThreads, 1) fp4_pair_kernel(const __grid_constant__ CUtensorMap tmW,
                                                                   const __grid_constant__ CUtensorMap tmX,
                                                                   const __grid_constant__ CUtensorMap tmSW,
                                                                   const __grid_constant__ CUtensorMap tmSX,
                                                                   const __grid_constant__ CUtensorMap tmOut,
                                                                   const Fp4ProductArgs args) {
    using C = PairCfg<FMT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* staged = smem + C::STAGES * C::STAGE_STRIDE;  // [half][2] pieces of the output
    float* terms = reinterpret_cast<float*>(staged + 4 * C::OUT_BYTES);  // of two tiles
    uint64_t* full = reinterpret_cast<uint64_t*>(terms + 4 * C::ROWS);
    uint64_t* empty = full + C::STAGES;
    uint64_t* tfull = empty + C::STAGES;
    uint64_t* handed = tfull + 2;  // the shared columns of a tile have been taken
    uint64_t* drain = handed + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&tfull[0], 1);
        mbar_init(&tfull[1], 1);
        mbar_init(handed, 2 * kEpilogue / 32);  // the epilogue warps of both CTAs
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
        prefetch_tensormap(&tmSW);
        prefetch_tensormap(&tmSX);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tc_fence_before();
    }
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are initialised before either arrives on the other's
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int n_wt = (args.N + 2 * kWRows - 1) / (2 * kWRows);
    const int n_tiles = n_wt * ((args.M + C::ROWS - 1) / C::ROWS);
    const int first = int(blockIdx.x) / 2, stride = int(gridDim.x) / 2;
    const int ktiles = (args.k64 + 3) / 4;
    griddep_wait();
    griddep_launch();

    if (warp == 0) {
        const uint32_t leader_full = cluster_map(smem_u32(full), 0);
        bool ok = true;
        int i = 0, s = 0;  // stages filled so far, and the next one
        uint32_t phase = 1;
        for (int t = first; ok && t < n_tiles; t += stride) {
            const int w0 = (t % n_wt) * 2 + int(rank), x0 = (t / n_wt) * 2;  // 128-row groups: own rows of w, x's first
            int sw = w0 * args.kgroups, sx = x0 * args.kgroups;              // scale groups of the K tile
            for (int kt = 0; kt < ktiles - args.withheld; ++kt, ++i) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[s], phase, abort_flag, args.flags, args.wait_ns));
                if (!ok) break;
                uint8_t* st = smem + s * C::STAGE_STRIDE;
                uint8_t* sc = st + kWBytes + C::X_BYTES;
                const uint32_t bar = leader_full + 8u * uint32_t(s);
                if (elect_one()) {
                    // rank 0's barrier counts the bytes of both CTAs
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE);
                    tma_load_2d_pair(st, &tmW, kt * kAtomBytes, w0 * kWRows, bar);
                    tma_load_2d_pair(st + kWBytes, &tmX, kt * kAtomBytes, (x0 + int(rank)) * kFp4RowGroup, bar);
                    tma_load_2d_pair(sc, &tmSW, 0, sw, bar);
                    tma_load_2d_pair(sc + C::S_BYTES, &tmSX, 0, sx, bar);
                    tma_load_2d_pair(sc + 2 * C::S_BYTES, &tmSX, 0, sx + args.kgroups, bar);
                }
                __syncwarp();
                sw += C::GROUPS;
                sx += C::GROUPS;
                if (++s == C::STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (args.withheld) break;
        }
        if (!ok && rank == 0) {  // let every copy that this CTA's barriers count land before it goes
            for (int j = i < C::STAGES ? 0 : i - C::STAGES; j < i; ++j)
                mbar_wait_bounded(&full[j % C::STAGES], uint32_t(j / C::STAGES & 1), nullptr, nullptr);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t peer_empty = cluster_map(smem_u32(empty), 1), peer_tfull = cluster_map(smem_u32(tfull), 1);
            const uint32_t sw = tmem + C::S_AT, sx = sw + 4 * C::GROUPS;
            const uint64_t d0 = smem_desc_sw128(smem_u32(smem)), c0 = scale_desc(smem_u32(smem) + kWBytes + C::X_BYTES);
            bool ok = true;
            int s = 0, j = 0;
            uint32_t phase = 0;
            for (int t = first; ok && t < n_tiles; t += stride, ++j) {
                const uint32_t acc = tmem + (j & 1 ? C::ACC1 : 0);
                if (j > 0) {  // the last tile's shared columns: whatever came before it has been read too
                    ok = mbar_wait_bounded(handed, uint32_t(j - 1) & 1u, abort_flag, args.flags, args.wait_ns, true);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                }
                for (int kt = 0; kt < ktiles; ++kt) {
                    ok = mbar_wait_bounded(&full[s], phase, abort_flag, args.flags, args.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t da = d0 + uint64_t(s * (C::STAGE_STRIDE >> 4)), db = da + (kWBytes >> 4);
                    const uint64_t dc = c0 + uint64_t(s * (C::STAGE_STRIDE >> 4));
                    const int nk = min(4, args.k64 - 4 * kt);
                    if (elect_one()) {
                        constexpr bool MX = FMT == CLEF_MXFP4;
                        auto copy = [&](uint32_t g) {
                            copy_scales<true>(sw + 4 * g, dc + g * (kFp4ScaleGroup >> 4));
                            copy_scales<true>(sx + 8 * g, dc + (C::GROUPS + g) * (kFp4ScaleGroup >> 4));
                            copy_scales<true>(sx + 8 * g + 4, dc + (2 * C::GROUPS + g) * (kFp4ScaleGroup >> 4));
                        };
                        copy(0);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t g = MX ? k / 2 : k;  // mxfp4: a group holds two MMAs' scales
                            if (MX ? k == 1 : k < 3) copy(g + 1);
                            if (k >= nk) continue;
                            mma_fp4<FMT, true>(acc, da + uint64_t(2 * k), db + uint64_t(2 * k),
                                               idesc_fp4(FMT, 2 * kWRows, C::ROWS, MX ? (k & 1) * 2 : 0), sw + 4 * g,
                                               sx + 8 * g, kt > 0 || k > 0 ? 1u : 0u);
                        }
                        tc_commit_pair(smem_u32(&empty[s]));  // the stage is free in both CTAs
                        tc_commit_pair(peer_empty + 8u * uint32_t(s));
                        if (kt == ktiles - 1) {
                            tc_commit_pair(smem_u32(&tfull[j & 1]));
                            tc_commit_pair(peer_tfull + 8u * uint32_t(j & 1));
                        }
                    }
                    __syncwarp();
                    if (++s == C::STAGES) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            // every MMA completes before TMEM is freed
            if (elect_one()) tc_commit_pair(smem_u32(drain));
            __syncwarp();
            mbar_wait_bounded(drain, 0, nullptr, args.flags);
        }
        __syncwarp();
    } else {
        const int tid = int(threadIdx.x) - 64;
        const int quarter = warp & 3, half = tid >> 7;  // TMEM lanes that this warp may read; its half of the columns
        const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
        const uint32_t leader_handed = cluster_map(smem_u32(handed), 0);
        // columns of the output that this thread writes: one, or four of the fragment form
        constexpr int NCOL = BULK ? 4 : 1;
        const int lane_n = int(rank) * kWRows + quarter * 32 + (BULK ? lane >> 2 : lane);
        // a tile's terms are read while the tile before it is written out
        float2 row = row_terms(args, first / n_wt * C::ROWS + tid);  // kEpilogue == ROWS
        ColumnTerms col[NCOL];
#pragma unroll
        for (int i = 0; i < NCOL; ++i) col[i] = column_terms(args, first % n_wt * 2 * kWRows + lane_n + 8 * i);
        // BULK: the half's two staged pieces in turn, each [2][16 rows][64 columns]
        uint8_t* piece = staged + half * 2 * C::OUT_BYTES;
        const uint32_t own = smem_u32(piece) + uint32_t(quarter >> 1) * (C::OUT_BYTES / 2) + uint32_t(lane & 7) * 128 +
                             uint32_t((((quarter & 1) * 4 + (lane >> 3)) ^ (lane & 7)) * 16);
        const bool issuer = (tid & 127) == 0;
        int j = 0;
        for (int t = first; t < n_tiles; t += stride, ++j) {
            const int m0 = t / n_wt * C::ROWS, n0 = t % n_wt * 2 * kWRows + int(rank) * kWRows;
            float* mine = terms + (j & 1) * 2 * C::ROWS;
            put_row_terms(mine, tid, row);
            const bool got = mbar_wait_bounded(&tfull[j & 1], uint32_t(j >> 1) & 1u, abort_flag, args.flags,
                                               args.wait_ns);
            tc_fence_after();
            // The accumulators share the last 64 columns of the first and the first 64 of the second: the
            // warps whose half they lie in take them and say so, the others only that they are done with the
            // tile before.
            const uint32_t acc = lanes + (j & 1 ? C::ACC1 : 0);
            const int c0 = half * 128, turn = half == 1 ? 64 : 0;  // half 1 takes its upper 64 columns first
            uint32_t r[2][32];
            auto take = [&](int at) {  // 64 columns
                if constexpr (BULK) {
                    tmem_ld16x64(acc + uint32_t(at), r[0]);
                    tmem_ld16x64(acc + uint32_t(at) + (16u << 16), r[1]);
                } else {
                    tmem_ld32(acc + uint32_t(at), r[0]);
                    tmem_ld32(acc + uint32_t(at + 32), r[1]);
                }
                tmem_ld_wait();
            };
            if (half != (j & 1)) {
                take(c0 + turn);
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(leader_handed);
            if (!epilogue_agrees(got)) break;  // all warps or none; the row terms are there too
            const int ahead = t + stride < n_tiles ? t + stride : t;
            ColumnTerms next[NCOL];
#pragma unroll
            for (int i = 0; i < NCOL; ++i) next[i] = column_terms(args, ahead % n_wt * 2 * kWRows + lane_n + 8 * i);
            row = row_terms(args, ahead / n_wt * C::ROWS + tid);
            const int rows = min(C::ROWS, args.M - m0);
#pragma unroll 1
            for (int c = 0; c < 128; c += 64) {
                const int at = c0 + (c ^ turn);
                if (c > 0 || half == (j & 1)) take(at);
                if constexpr (BULK) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        // a piece is written while the other is read; before the barrier of one, the other has been
                        const uint32_t to = own + (q & 1) * C::OUT_BYTES;
                        const float* tq = mine + 2 * (at + 16 * q);
                        if (q == 0) stage16<OUT, 0>(to, r[0], r[1], col, tq, lane);
                        if (q == 1) stage16<OUT, 8>(to, r[0], r[1], col, tq, lane);
                        if (q == 2) stage16<OUT, 16>(to, r[0], r[1], col, tq, lane);
                        if (q == 3) stage16<OUT, 24>(to, r[0], r[1], col, tq, lane);
                        fence_proxy_async_smem();
                        if (issuer) bulk_wait_read<0>();
                        half_sync(half);
                        if (issuer && at + 16 * q < rows) {
                            const uint8_t* from = piece + (q & 1) * C::OUT_BYTES;
                            if (n0 < args.N) tma_store_2d(&tmOut, from, n0, m0 + at + 16 * q);
                            if (n0 + 64 < args.N) tma_store_2d(&tmOut, from + C::OUT_BYTES / 2, n0 + 64, m0 + at + 16 * q);
                            bulk_commit();
                        }
                    }
                } else {
                    if (at < rows) emit<OUT, 32>(args, r[0], col[0], mine + 2 * at, m0 + at, rows - at, n0 + quarter * 32 + lane, lane);
                    if (at + 32 < rows)
                        emit<OUT, 32>(args, r[1], col[0], mine + 2 * at + 64, m0 + at + 32, rows - at - 32,
                                      n0 + quarter * 32 + lane, lane);
                }
            }
#pragma unroll
            for (int i = 0; i < NCOL; ++i) col[i] = next[i];
            tc_fence_before();
        }
        if (BULK && issuer) bulk_wait_all();
    }
    __syncthreads();
    // no CTA leaves (or frees TMEM) while the other's MMAs, copies or arrivals may still touch it
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// Pairs that the current device holds at once, found out once for every device.
template <int FMT, int OUT, bool BULK>
cudaError_t pairs_at_once(int* n) {
    using C = PairCfg<FMT>;
    static PerDevice<int> known;
    int device = 0;
    const cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    return cudaError_t(known.get(device, n, [](int* v) {
        cudaError_t f = cudaFuncSetAttribute(fp4_pair_kernel<FMT, OUT, BULK>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (f != cudaSuccess) return int(f);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = C::SMEM;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        f = cudaOccupancyMaxActiveClusters(v, fp4_pair_kernel<FMT, OUT, BULK>, &cfg);
        return f != cudaSuccess ? int(f) : *v < 1 ? int(cudaErrorInvalidConfiguration) : 0;
    }));
}

template <int FMT, int OUT, bool BULK>
cudaError_t launch_pair(const clef_fp4& x, const clef_fp4& w, const Fp4ProductArgs& a, cudaStream_t s) {
    using C = PairCfg<FMT>;
    int pairs = 0;
    const cudaError_t e = pairs_at_once<FMT, OUT, BULK>(&pairs);
    if (e != cudaSuccess) return e;
    CUtensorMap maps[5];
    if (!codes_map(&maps[0], w, kWRows) || !codes_map(&maps[1], x, C::ROWS / 2) || !scales_map(&maps[2], w) ||
        !scales_map(&maps[3], x))
        return cudaErrorInvalidValue;
    maps[4] = maps[0];  // a map that is never used where the output is not stored by TMA
    if (BULK && !make_tma_2d(&maps[4], a.out, 2, uint64_t(a.N), uint64_t(a.M), uint64_t(a.ldo) * 2, 64, 16, true))
        return cudaErrorInvalidValue;
    const int tiles = (a.N + 2 * kWRows - 1) / (2 * kWRows) * ((a.M + C::ROWS - 1) / C::ROWS);
    return launch_clusters(fp4_pair_kernel<FMT, OUT, BULK>, 2 * std::min(tiles, pairs), 2, kThreads, C::SMEM, s, maps, a);
}

template <int FMT, int OUT>
cudaError_t launch_product(const clef_fp4& x, const clef_fp4& w, const Fp4ProductArgs& a, cudaStream_t s) {
    // Tiles of 128 x 128 while two of them at most fall to an SM (one, where K is long: then pairs, which load
    // half as much, win); measured on both sides at N 1024 to 16384, K 512 to 16384:
    //   4096 x 4096, 1024 rows (256 tiles): tiles 10.7 us, pairs 10.8; 1280 rows (320): 18.6, 15.3
    //   4096 x 1024, 1024 rows: 6.2, 7.4; 1280 rows: 10.5, 9.9
    //   4096 x 16384, 512 rows (128 tiles): 22.9, 23.2; 608 rows (160): 27.6, 23.5
    const int64_t tiles = int64_t((a.N + kWRows - 1) / kWRows) * ((a.M + 127) / 128);
    if (a.M > 64 && tiles > (fp4_ktiles(x.cols) > 16 ? 1 : 2) * num_sms()) {
        if constexpr (OUT != CLEF_FP32)
            if (a.bulk) return launch_pair<FMT, OUT, true>(x, w, a, s);
        return launch_pair<FMT, OUT, false>(x, w, a, s);
    }
    if (a.M <= 32) return launch_tile<FMT, 32, OUT, kKept>(&x, w, a, s);
    if (a.M <= 64) return launch_tile<FMT, 64, OUT, kKept>(&x, w, a, s);
    return launch_tile<FMT, 128, OUT, kKept>(&x, w, a, s);
}

}  // namespace

cudaError_t launch_fp4_product(const clef_fp4& x, const clef_fp4& w, const Fp4ProductArgs& a, int dtype,
                               cudaStream_t s) {
    if (x.format == CLEF_MXFP4) {
        if (dtype == CLEF_BF16) return launch_product<CLEF_MXFP4, CLEF_BF16>(x, w, a, s);
        if (dtype == CLEF_FP16) return launch_product<CLEF_MXFP4, CLEF_FP16>(x, w, a, s);
        return launch_product<CLEF_MXFP4, CLEF_FP32>(x, w, a, s);
    }
    if (dtype == CLEF_BF16) return launch_product<CLEF_NVFP4, CLEF_BF16>(x, w, a, s);
    if (dtype == CLEF_FP16) return launch_product<CLEF_NVFP4, CLEF_FP16>(x, w, a, s);
    return launch_product<CLEF_NVFP4, CLEF_FP32>(x, w, a, s);
}

}  // namespace clef
