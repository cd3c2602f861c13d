// Attention over the paged 4-bit memory cache (clef_cache_attend).
//
// The few-rows kernel, and the merge of both kernels' splits; cache_attend_rows.cu has the
// kernel for requests of many query rows.
//
// A CTA of four warps takes one item: a split of a request's keys, one key/value head, and up
// to 4 C NT query rows of the heads that share it.  Its warps take the split in steps of 32
// keys (two 16-token pieces) in turn, each through a ring of its own that cp.async fills
// several steps ahead (no barrier, nothing to wait for but the warp's own copies), and meet at
// the end of the item to weigh their results; the next item's pages, pieces and queries are
// under way by then.  The products run transposed on mma.sync, the keys as the M dimension:
// S^T = K Q^T (16 keys x 8 queries an instruction, so that a single token wastes 7 of 8 columns
// rather than 15 of 16 rows) and O^T += V^T P^T.  The A operand of both is made in registers
// from the codes: the stored order gives each lane its own 16 bytes of a 16-token piece.
//   Keys: a 4-bit code in bits 0-3 of an fp16 word is the subnormal c 2^-24, exact, and in
// bits 4-7 c 2^-20, so one AND makes two operand values; the 2^4 between the two halves of
// a run of 16 is taken out of the queries instead.  The score is then, in fp32,
//   s_t (q . c_t) + m_t (sum q),  with s_t and m_t the key's scale and minimum.
// Queries are scaled by a power of two per row to fill fp16's range (exact).
//   Values: with w_t = p_t s_t,
//   o = sum_t p_t (s_t c_t + m_t) = sum_t w_t c_t - sum_t 8 w_t + sum_t p_t (m_t + 8 s_t).
// The weights w_t are rounded to fp16 (11 bits; after a power of two of the row's own, see
// move_weights in cache_attend.cuh), once for the first two sums, which are products
// of the matrix unit with the codes and with eights: their difference is that of centred codes
// |c - 8| <= 8, and what the rounding costs is relative to it, not to the whole range of the
// codes.  The third sum is fp32.  An fp16 output keeps as many digits as the weights, so for fp16
// (FINE) what the rounding leaves of a weight is rounded to fp16 too and multiplied after it: 22 bits.
// There the codes are centred: the matrix unit's additions round towards zero, so a difference of
// two large sums would be off by 2^-19 of them, always to the same side.  (Centring the codes
// takes 16 more instructions a piece; that and the second product make fp16 17 % slower: 61 us
// against 52 for a decoding step of 64 requests with 8 heads of 128.)
// The softmax reference of a row moves only when a score exceeds it by 2^8 (then all sums
// of the warp are rescaled), so that a step needs no reduction between lanes: each lane sums
// the keys that it holds, and the lanes are added once at the end of the item.
//
// Requests longer than one split leave normalised partials with their log-sum, which the
// merge kernel weighs.
//
// What bounds it: instruction issue, the integer pipe above all (about 142 instructions for 16
// keys of 64 values, 40 of them to split codes; 52 % of the issue slots and 57 % of the memory rate
// in a decoding step of 64 requests of 156 to 16384 keys with 8 heads of 128: 218 MB in 52 us),
// and the unequal ends of a call; 256 requests of 4096 keys (1.2 GB) take 216 us, 83 % of the
// memory's measured copy rate.
#include "cache_attend.cuh"

namespace clef {

template <int G, int NT, int C>
struct AttendSmem {
    // 16-token pieces a step: two halve the cost of a step's waits, votes and addresses; the same
    // for all, so that a row's sums do not depend on the other requests' rows
    static constexpr int kPieces = 2;
    // steps in flight a warp
    static constexpr int kStages = G == 2 ? 2 : NT <= 2 ? 3 : 4;
    static constexpr int kRing = kAttendWarps * kStages * kPieces * kPiece * G;
    static constexpr int kRows = 4 * C * NT;  // query rows of an item
    static constexpr int kResults = kAttendWarps * kRows * 64 * G * 4;  // the warps' sums of values
    static constexpr int kBytes = kRing + kResults + 2 * kAttendWarps * kRows * 4;
};

template <int G, int NT, int C, bool FINE>
__global__ void __launch_bounds__(kAttendThreads, G == 2 ? (NT == 1 ? 3 : 2) : NT == 1 ? 4 : NT == 2 ? 3 : 2)
    cache_attend_kernel(const CacheAttendArgs a) {
    using Smem = AttendSmem<G, NT, C>;
    constexpr int ST = Smem::kStages, KP = Smem::kPieces;
    constexpr int kBytes = kPiece * G, R = Smem::kRows;
    // column c of a lane's in block n is row `row_of(n, c)` of the item
    auto row_of = [&](int n, int c) { return C == 2 ? n * 8 + 2 * (int(threadIdx.x) & 3) + c : int(threadIdx.x) & 3; };
    constexpr int kMaxPages = kAttendMaxChunk / 16;
    griddep_wait();
    griddep_launch();
    extern __shared__ __align__(16) uint8_t smem[];
    float* results = reinterpret_cast<float*>(smem + Smem::kRing);  // [warp][row][value]
    float* s_ref = results + Smem::kResults / 4;                     // [warp][row]
    float* s_sum = s_ref + kAttendWarps * R;
    const Requests s_req(reinterpret_cast<int*>(smem + Smem::kBytes), a.B);
    __shared__ int s_page[2][kMaxPages];  // page numbers of the split at hand and of the next one
    const int n_items = scan_requests<G, false>(a, s_req, R);
    if (blockIdx.x == 0 && a.part_off)
        for (int b = threadIdx.x; b < a.B; b += kAttendThreads) a.part_off[b] = b ? s_req.parts[b - 1] : 0;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, tq = lane & 3;
    const int page_mask = a.c.page - 1;
    uint8_t* ring = smem + warp * (ST * KP * kBytes);
    constexpr int kStride = 16 * KP * kAttendWarps;

    // Items run into one another: while the pieces of one are worked off, the next one's page
    // numbers arrive; its first pieces and queries are requested before the results of the
    // first are weighed.
    auto request_pages = [&](const Item& k, int* to) {
        for (int i = threadIdx.x; i < kMaxPages; i += kAttendThreads)
            if ((int64_t(k.p0 + i) << a.c.page_shift) < k.t1)
                cp_async4(to + i, a.table + int64_t(k.b) * a.width + k.p0 + i);
    };
    // does the item lack a page? (all lanes of the warp get the answer)
    auto lacks_pages = [&](const Item& k, const int* pages) {
        bool bad = false;
#pragma unroll
        for (int i = lane; i < kMaxPages; i += 32)
            if ((int64_t(k.p0 + i) << a.c.page_shift) < k.t1) bad |= pages[i] < 0 || pages[i] >= a.c.n_pages;
        if (bad) atomicOr(a.flags, kFlagBounds);
        return bool(__any_sync(0xffffffffu, bad));
    };
    auto piece_at = [&](const Item& k, const int* pages, int t) -> const uint8_t* {
        const int id = pages[(t >> a.c.page_shift) - k.p0];
        if (id < 0 || id >= a.c.n_pages) return nullptr;
        return a.c.data + (((int64_t(id) * a.c.heads + a.head0 + k.h) << (a.c.page_shift - 4)) + ((t & page_mask) >> 4)) * kBytes;
    };
    // pages of 32 tokens and more hold a step's pieces side by side (what lies behind the
    // last token is never used)
    auto request_step = [&](const Item& k, const int* pages, int t, int stage) {
        if (t < k.t1) {
            uint8_t* dst = ring + stage * (KP * kBytes) + lane * 16;
            if (a.c.page_shift > 4) {
                const uint8_t* src = piece_at(k, pages, t);
                if (src)
#pragma unroll
                    for (int i = 0; i < KP * kBytes; i += 512)
                        if (i + lane * 16 < KP * kBytes) cp_async16(dst + i, src + lane * 16 + i, true);
            } else {
#pragma unroll
                for (int j = 0; j < KP; ++j) {
                    const uint8_t* src = t + 16 * j < k.t1 ? piece_at(k, pages, t + 16 * j) : nullptr;
                    if (src)
#pragma unroll
                        for (int i = 0; i < kBytes; i += 512)
                            if (i + lane * 16 < kBytes) cp_async16(dst + j * kBytes + i, src + lane * 16 + i, true);
                }
            }
        }
        cp_async_commit();
    };
    auto request_first = [&](const Item& k, const int* pages) {
#pragma unroll
        for (int s = 0; s < ST - 1; ++s) request_step(k, pages, k.t0 + warp * 16 * KP + s * kStride, s);
    };
    // a lane's query words: rows g of each block of 8, values 2 tq, 2 tq + 1 of each run of 8
    auto load_queries = [&](const Item& k, uint32_t (&qw)[NT][G][8]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = C == 2 ? n * 8 + g : g >> 1;
            const bool live = r < k.rows && (C == 2 || !(g & 1));
            const int qi = live ? a.by_share(k.row0 + r) : 0;
            const int qh = k.h * a.share + (live ? k.row0 + r - qi * a.share : 0);
            const uint16_t* q = static_cast<const uint16_t*>(a.q) + (s_req.q0[k.b] + qi) * a.q_row + qh * a.q_head + 2 * tq;
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    qw[n][gr][i] = live ? __ldg(reinterpret_cast<const uint32_t*>(q + gr * 64 + i * 8)) : 0u;
        }
    };

    if (item_of_turn(0) >= n_items) return;
    Item me = item_of<R>(a, s_req, item_of_turn(0));
    request_pages(me, s_page[0]);
    cp_async_commit();
    uint32_t qw[NT][G][8];
    load_queries(me, qw);
    cp_async_wait<0>();
    __syncthreads();
    request_first(me, s_page[0]);

    for (int turn = 0;; ++turn) {
        const int* pages = s_page[turn & 1];
        const int t0 = me.t0, t1 = me.t1, ahead = me.ahead;
        const bool holes = lacks_pages(me, pages);

        // ---- queries: B operand of S^T, one row a group of four lanes
        uint32_t qf[G][NT][8];
        float qscale[NT][2], qsum[G][NT][2];  // of rows 2 tq, 2 tq + 1 of each block of 8
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float2 x[G][8];
            float top = 0.f, sum[G];
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                sum[gr] = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[gr][i] = unpack2(qw[n][gr][i], a.dtype);
                    sum[gr] += x[gr][i].x + x[gr][i].y;
                    top = fmaxf(top, fmaxf(fabsf(x[gr][i].x), fabsf(x[gr][i].y)));
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], o);
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            // the row's largest value goes to [2^14, 2^15)
            const int e = top > 0.f ? 14 - (int(__float_as_uint(top) >> 23) - 127) : 0;
            const float up = pow2i(min(e, 120));
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float f = (i & 1) ? up * 0.0625f : up;
                    qf[gr][n][i] = pack_f16(x[gr][i].x * f, x[gr][i].y * f);
                }
            const float back = a.scale_log2 * pow2i(24 - min(e, 120));
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int from = (2 * tq + c) * 4;
                qscale[n][c] = __shfl_sync(0xffffffffu, back, from);
#pragma unroll
                for (int gr = 0; gr < G; ++gr)
                    qsum[gr][n][c] = __shfl_sync(0xffffffffu, sum[gr], from) * a.scale_log2;
            }
        }

        float acc[G][4][NT][4];  // O^T: 4 blocks of 16 values of each group
        float mid[G][NT][4];     // eight times the sum of the weights, as acc counts
        float l[NT][2], z[G][NT][2], ref[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                l[n][c] = 0.f;
                ref[n][c] = 0.f;
#pragma unroll
                for (int gr = 0; gr < G; ++gr) z[gr][n][c] = mid[gr][n][c] = mid[gr][n][c + 2] = 0.f;
            }
#pragma unroll
        for (int gr = 0; gr < G; ++gr)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[gr][mt][n][c] = 0.f;
        float mul[G][NT][2];  // the weights' powers of two
#pragma unroll
        for (int gr = 0; gr < G; ++gr)
#pragma unroll
            for (int n = 0; n < NT; ++n) mul[gr][n][0] = mul[gr][n][1] = 1.f;
        bool first = true;  // no step yet: the references are still to be set

        // the next item's page numbers come in with the pieces of this one
        const int w_next = item_of_turn(turn + 1);
        const bool more = w_next < n_items;
        Item next = me;
        if (more) {
            next = item_of<R>(a, s_req, w_next);
            request_pages(next, s_page[~turn & 1]);
        }

        int stage = 0;
        for (int t = t0 + warp * 16 * KP; t < t1; t += kStride) {
            cp_async_wait<ST - 2>();
            __syncwarp();  // this step's pieces are there, and every lane is done with those before
            request_step(me, pages, t + (ST - 1) * kStride, stage == 0 ? ST - 1 : stage - 1);
            const uint8_t* pieces = ring + stage * (KP * kBytes);
            stage = stage == ST - 1 ? 0 : stage + 1;

            // ---- key products, scales and minima (keys g and g + 8 of each piece)
            float part[KP][G][NT][4];
            float ks[KP][G][2], km[KP][G][2], vs[KP][G][2], vm[KP][G][2];
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    const uint8_t* piece = pieces + k * kBytes;
                    const uint4 kw = reinterpret_cast<const uint4*>(piece + gr * 512)[lane];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint2 sm = *reinterpret_cast<const uint2*>(piece + G * 1024 + ((g + 8 * r) * G + gr) * 8);
                        ks[k][gr][r] = bf16_lo(sm.x);
                        km[k][gr][r] = bf16_hi(sm.x);
                        vs[k][gr][r] = bf16_lo(sm.y);
                        vm[k][gr][r] = bf16_hi(sm.y);
                    }
                    const uint32_t words[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t x = words[i], y = x >> 8;
                        const uint32_t A[4] = {x & 0x000F000Fu, y & 0x000F000Fu, x & 0x00F000F0u, y & 0x00F000F0u};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (i == 0)
                                mma_f16_16816_first(part[k][gr][n], A, qf[gr][n][0], qf[gr][n][1]);
                            else
                                mma_f16_16816(part[k][gr][n], A, qf[gr][n][2 * i], qf[gr][n][2 * i + 1]);
                        }
                    }
                }
            // ---- scores (base 2) less their row's reference
            float p[KP][NT][4], top = -INFINITY;
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; c += 3 - C) {
                        float y = -ref[n][c & 1];
#pragma unroll
                        for (int gr = 0; gr < G; ++gr) {
                            y = fmaf(qsum[gr][n][c & 1], km[k][gr][c >> 1], y);
                            y = fmaf(part[k][gr][n][c] * qscale[n][c & 1], ks[k][gr][c >> 1], y);
                        }
                        p[k][n][c] = y;
                    }
            // tokens behind the last one hold anything, causal rows see a part, pages may lack
            if (t + 16 * KP > t1 || (a.causal && t + 16 * KP - 1 > ahead) || holes) {
                bool odd = false, any = false;  // a value scale that is no number; a token that is there
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    const int tk = t + 16 * k;
                    const int end = tk < t1 && piece_at(me, pages, tk) ? t1 : 0;
                    any |= tk < end;
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (tk + g + 8 * r >= end)
#pragma unroll
                            for (int gr = 0; gr < G; ++gr) vs[k][gr][r] = vm[k][gr][r] = 0.f;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 4; c += 3 - C) {
                            const int sees = a.causal ? ahead + a.by_share(me.row0 + row_of(n, c & 1)) + 1 : end;
                            if (tk + g + 8 * (c >> 1) >= min(sees, end)) p[k][n][c] = -INFINITY;
                        }
#pragma unroll
                    for (int gr = 0; gr < G; ++gr)
#pragma unroll
                        for (int r = 0; r < 2; ++r) odd |= !(fabsf(vs[k][gr][r]) < INFINITY);
                }
                if (first && !any) continue;
                if (odd) {  // it makes the rows that see it no number, and is nothing to the others
#pragma unroll
                    for (int k = 0; k < KP; ++k)
#pragma unroll
                        for (int gr = 0; gr < G; ++gr)
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                if (!(fabsf(vs[k][gr][r]) < INFINITY)) {
                                    vs[k][gr][r] = vm[k][gr][r] = 0.f;
#pragma unroll
                                    for (int n = 0; n < NT; ++n)
#pragma unroll
                                        for (int c = 0; c < C; ++c)
                                            if (!(p[k][n][c + 2 * r] == -INFINITY)) z[gr][n][c] = NAN;
                                }
                }
            }
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (C == 2) {
                        top = fmax3(top, p[k][n][0], p[k][n][1]);
                        top = fmax3(top, p[k][n][2], p[k][n][3]);
                    } else {
                        top = fmax3(top, p[k][n][0], p[k][n][2]);
                    }
                }
            if (__any_sync(0xffffffffu, first || top > 8.f)) {  // new references: the first step, and rarely after
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        float mx = -INFINITY;  // relative to the reference (0 in the first step)
#pragma unroll
                        for (int k = 0; k < KP; ++k) mx = fmax3(mx, p[k][n][c], p[k][n][c + 2]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        const bool moved = first ? mx > -INFINITY : mx > 8.f;
                        Decay d;
                        if (moved) {
                            if (!first) d.set(mx);
                            ref[n][c] += mx;
                            l[n][c] *= d.corr;
#pragma unroll
                            for (int k = 0; k < KP; ++k) {
                                p[k][n][c] -= mx;
                                p[k][n][c + 2] -= mx;
                            }
                        }
#pragma unroll
                        for (int gr = 0; gr < G; ++gr) {
                            float x = 0.f, big = 0.f;
#pragma unroll
                            for (int k = 0; k < KP; ++k)
                                x = fmax3(x, ex2_approx(p[k][n][c]) * vs[k][gr][0], ex2_approx(p[k][n][c + 2]) * vs[k][gr][1]);
#pragma unroll
                            for (int mt = 0; mt < 4; ++mt)
                                big = fmax3(big, fabsf(acc[gr][mt][n][c]), fabsf(acc[gr][mt][n][c + 2]));
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) {
                                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                            }
                            if (moved) {
                                const float f = move_weights(mul[gr][n][c], x, big, d);
                                z[gr][n][c] *= d.corr;
                                mid[gr][n][c] *= f;
                                mid[gr][n][c + 2] *= f;
#pragma unroll
                                for (int mt = 0; mt < 4; ++mt) {
                                    acc[gr][mt][n][c] *= f;
                                    acc[gr][mt][n][c + 2] *= f;
                                }
                            }
                        }
                    }
                first = false;
            }
            // ---- weights
            uint32_t pf[KP][G][NT][2], pl[KP][G][NT][2];  // FINE: pl holds what rounding left of pf
            float most = 0.f;
            auto weigh = [&](int k, int gr, int n, int r) {
                float w[2] = {0.f, 0.f};
#pragma unroll
                for (int c = 0; c < C; ++c) w[c] = p[k][n][2 * r + c] * mul[gr][n][c] * vs[k][gr][r];
                pf[k][gr][n][r] = pack_f16(w[0], w[1]);
                if (FINE) pl[k][gr][n][r] = rest_f16(pf[k][gr][n][r], w[0], w[1]);
                return C == 2 ? fmaxf(w[0], w[1]) : w[0];
            };
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int c = 0; c < 4; c += 3 - C) {
                        p[k][n][c] = ex2_approx(p[k][n][c]);
                        l[n][c & 1] += p[k][n][c];
                    }
#pragma unroll
                    for (int gr = 0; gr < G; ++gr)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float mid_value = fmaf(8.f, vs[k][gr][r], vm[k][gr][r]);
#pragma unroll
                            for (int c = 0; c < C; ++c) z[gr][n][c] = fmaf(p[k][n][2 * r + c], mid_value, z[gr][n][c]);
                            most = fmaxf(most, weigh(k, gr, n, r));
                        }
                }
            if (__any_sync(0xffffffffu, most > kMostWeight)) {  // larger values than the rows have used before
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            float x = 0.f;
#pragma unroll
                            for (int k = 0; k < KP; ++k)
                                x = fmax3(x, p[k][n][c] * vs[k][gr][0], p[k][n][c + 2] * vs[k][gr][1]);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                            if (x * mul[gr][n][c] > kMostWeight) {
                                const float f = move_weights(mul[gr][n][c], x, 0.f, Decay());
                                mid[gr][n][c] *= f;
                                mid[gr][n][c + 2] *= f;
#pragma unroll
                                for (int mt = 0; mt < 4; ++mt) {
                                    acc[gr][mt][n][c] *= f;
                                    acc[gr][mt][n][c + 2] *= f;
                                }
                            }
                        }
#pragma unroll
                        for (int k = 0; k < KP; ++k)
#pragma unroll
                            for (int r = 0; r < 2; ++r) weigh(k, gr, n, r);
                    }
            }
            // ---- value products
#pragma unroll
            for (int k = 0; k < KP; ++k)
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    const uint4 codes = reinterpret_cast<const uint4*>(pieces + k * kBytes + (G + gr) * 512)[lane];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            pf[k][gr][n][r] = transpose8(pf[k][gr][n][r]);
                            if (FINE) pl[k][gr][n][r] = transpose8(pl[k][gr][n][r]);
                        }
                    const uint32_t words[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) {
                        const uint32_t x = words[mt], y = x >> 8;
                        const uint32_t A[4] = {FINE ? centred_low(x) : x & 0x000F000Fu, FINE ? centred_high(x) : x & 0x00F000F0u,
                                               FINE ? centred_low(y) : y & 0x000F000Fu, FINE ? centred_high(y) : y & 0x00F000F0u};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_f16_16816(acc[gr][mt][n], A, pf[k][gr][n][0], pf[k][gr][n][1]);
                            if (FINE) mma_f16_16816(acc[gr][mt][n], A, pl[k][gr][n][0], pl[k][gr][n][1]);
                        }
                    }
                    if (FINE) continue;
                    constexpr uint32_t kEights[4] = {0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u};
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16_16816(mid[gr][n], kEights, pf[k][gr][n][0], pf[k][gr][n][1]);
                }
        }
        cp_async_commit();  // page numbers, where the warp had no step
        cp_async_wait<0>();

        // ---- the warps' results side by side in shared memory, then weighed: normalised, with
        // the logarithm (base 2) of the sum
        __syncthreads();  // the results of the item before this one are no longer read
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float sum = l[n][c], zs[G];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    zs[gr] = z[gr][n][c];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) zs[gr] += __shfl_xor_sync(0xffffffffu, zs[gr], o);
                }
                const int r = row_of(n, c);
                if (g == 0) {
                    s_ref[warp * R + r] = sum == 0.f ? -1e30f : ref[n][c];
                    s_sum[warp * R + r] = sum;
                }
                float* dst = results + (warp * R + r) * (64 * G);
#pragma unroll
                for (int gr = 0; gr < G; ++gr)
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                        for (int half = 0; half < 2; ++half)
                            // (codes of the upper half of a run count 2^4, and all 2^-24)
                            dst[gr * 64 + mt * 16 + half * 8 + g] =
                                FINE ? fmaf(acc[gr][mt][n][c + 2 * half], 1.f / mul[gr][n][c], zs[gr]) :
                                fmaf(0x1p24f * fmaf(acc[gr][mt][n][c + 2 * half], half ? 0.0625f : 1.f,
                                                    -mid[gr][n][c + 2 * half]),
                                     1.f / mul[gr][n][c], zs[gr]);
            }
        __syncthreads();  // the results and the next item's page numbers are there
        if (more) {
            request_first(next, s_page[~turn & 1]);
            load_queries(next, qw);
        }
        const bool whole = s_req.len[me.b] <= a.chunk;
        // warp w finishes rows w, w + 4, ...: lane i weighs the i-th of them, then all lanes its values
        float wgt[kAttendWarps];
        int64_t row = -1;
        if (lane < C * NT) {
            const int r = warp + kAttendWarps * lane;
            float top = -1e30f, sum = 0.f;
#pragma unroll
            for (int i = 0; i < kAttendWarps; ++i) top = fmaxf(top, s_ref[i * R + r]);
#pragma unroll
            for (int i = 0; i < kAttendWarps; ++i) {
                wgt[i] = ex2_approx(s_ref[i * R + r] - top);
                sum = fmaf(s_sum[i * R + r], wgt[i], sum);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int i = 0; i < kAttendWarps; ++i) wgt[i] *= inv;
            if (r < me.rows) {
                const int qi = a.by_share(me.row0 + r), qh = me.h * a.share + me.row0 + r - qi * a.share;
                row = whole ? int64_t(s_req.q0[me.b] + qi) * a.q_heads + qh
                            : (me.b ? s_req.parts[me.b - 1] : 0) + (int64_t(me.split) * s_req.nq[me.b] + qi) * a.q_heads + qh;
                // (query rows of requests that overlap, which cu_q must not have, could make
                // more partial rows than the workspace holds)
                if (!whole && (row < 0 || row >= a.part_rows)) {
                    atomicOr(a.flags, kFlagBounds);
                    row = -1;
                }
                const float lse2 = sum == 0.f ? -INFINITY : top + log2f(sum);
                if (row >= 0 && !whole) a.part_lse[row] = lse2;
                if (whole && a.lse) a.lse[row] = lse2 * 0.6931471805599453f;
            }
        }
#pragma unroll
        for (int j = 0; j < C * NT; ++j) {
            const int64_t to = __shfl_sync(0xffffffffu, row, j);
            float wj[kAttendWarps];
#pragma unroll
            for (int i = 0; i < kAttendWarps; ++i) wj[i] = __shfl_sync(0xffffffffu, wgt[i], j);
            if (to < 0) continue;
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                float2 o = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kAttendWarps; ++i) {
                    const float2 x = *reinterpret_cast<const float2*>(results + (i * R + warp + kAttendWarps * j) * (64 * G) +
                                                                      gr * 64 + lane * 2);
                    o.x = fmaf(x.x, wj[i], o.x);
                    o.y = fmaf(x.y, wj[i], o.y);
                }
                const int64_t at = to * (64 * G) + gr * 64 + lane * 2;
                if (!whole)
                    *reinterpret_cast<float2*>(a.part_o + at) = o;
                else
                    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at) =
                        a.dtype == 0 ? pack_bf16(o.x, o.y) : pack_f16(o.x, o.y);
            }
        }
        if (!more) return;
        me = next;
    }
}

// Some splits of a row, weighed: the largest log-sum, the sum of weights and values relative to it.
template <int G>
struct Weighed {
    float top, sum, o[2 * G];
    __device__ void clear() {
        top = -1e30f;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) o[i] = 0.f;
    }
};

// Splits k0 .. k0 + 7 of the n of a row (all their loads under way at once), added to `x`.
template <int G>
__device__ __forceinline__ void weigh_eight(const CacheAttendArgs& a, int64_t p0, int64_t stride, int k0, int n, Weighed<G>& x) {
    const int lane = threadIdx.x & 31;
    n = min(8, n - k0);
    const float y = lane < n ? a.part_lse[p0 + (k0 + lane) * stride] : -INFINITY;
    float2 v[8][G];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < G; ++i)
            v[j][i] = j < n ? *reinterpret_cast<const float2*>(a.part_o + (p0 + (k0 + j) * stride) * (64 * G) + i * 64 + lane * 2)
                            : make_float2(0.f, 0.f);
    const float mx = fmaxf(x.top, warp_max(y));
    const float corr = ex2_approx(x.top - mx), w = ex2_approx(y - mx);
    x.sum = fmaf(x.sum, corr, warp_sum(w));
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) x.o[i] *= corr;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            x.o[2 * i] = fmaf(v[j][i].x, wj, x.o[2 * i]);
            x.o[2 * i + 1] = fmaf(v[j][i].y, wj, x.o[2 * i + 1]);
        }
    }
    x.top = mx;
}

// `x` added to `all`, whose top is the largest of all that are added.
template <int G>
__device__ __forceinline__ void add_weighed(Weighed<G>& all, const Weighed<G>& x) {
    const float w = ex2_approx(x.top - all.top);
    all.sum = fmaf(x.sum, w, all.sum);
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) all.o[i] = fmaf(x.o[i], w, all.o[i]);
}

// Weighs the splits of one (query row, head), two values of each group a lane.  The splits form
// eight parts, eight splits in turn each (0-7 and 64-71 are the first part's), and the parts are
// added in their order: the same sums in both forms, whatever the other requests' lengths are.  WIDE:
// a CTA's eight warps take a part each and meet in shared memory; otherwise (16 splits at most, so two
// parts) each warp has a row of its own.
template <int G, bool WIDE>
__global__ void __launch_bounds__(256) cache_merge_kernel(const CacheAttendArgs a) {
    griddep_wait();
    griddep_launch();
    __shared__ Weighed<G> s_part[8][WIDE ? 32 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.y;
    const int64_t item = WIDE ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * 8 + warp;
    const Request r = request_of(a, b, false);
    const int64_t p0 = a.part_off[b] + item, stride = int64_t(r.nq) * a.q_heads;
    // a row of a request of one split is finished; one outside the workspace has been reported
    const bool live = r.chunks > 1 && item < stride && p0 >= 0 && p0 + (r.chunks - 1) * stride < a.part_rows;
    const int chunks = live ? r.chunks : 0;
    Weighed<G> all;
    all.clear();
    if (WIDE) {  // (a CTA without a row goes through it empty)
        const int n_parts = min(8, (chunks + 7) / 8);
        if (warp < n_parts) {
            Weighed<G> mine;
            mine.clear();
            for (int k0 = warp * 8; k0 < chunks; k0 += 64) weigh_eight<G>(a, p0, stride, k0, chunks, mine);
            s_part[warp][lane] = mine;
        }
        __syncthreads();
        if (warp != 0) return;
        for (int j = 0; j < n_parts; ++j) all.top = fmaxf(all.top, s_part[j][lane].top);
        for (int j = 0; j < n_parts; ++j) add_weighed<G>(all, s_part[j][lane]);
    } else {
        Weighed<G> part[2];
        part[0].clear();
        part[1].clear();
        if (chunks > 0) weigh_eight<G>(a, p0, stride, 0, chunks, part[0]);
        if (chunks > 8) weigh_eight<G>(a, p0, stride, 8, chunks, part[1]);
        all.top = fmaxf(part[0].top, part[1].top);
        add_weighed<G>(all, part[0]);
        if (chunks > 8) add_weighed<G>(all, part[1]);
    }
    if (!live) return;  // (at the end: warps that leave at once made the call of 64 single tokens 65 us, not 52)
    const float top = all.top, sum = all.sum, (&o)[2 * G] = all.o;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t row = int64_t(r.q0) * a.q_heads + item;
    if (lane == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row * (64 * G)) + lane;
#pragma unroll
    for (int i = 0; i < G; ++i)
        out[i * 32] = a.dtype == 0 ? pack_bf16(o[2 * i] * inv, o[2 * i + 1] * inv) : pack_f16(o[2 * i] * inv, o[2 * i + 1] * inv);
}

namespace {

template <int G, int NT, int C, bool FINE>
cudaError_t launch_attend_as(const CacheAttendArgs& a, cudaStream_t s) {
    constexpr int kBytes = AttendSmem<G, NT, C>::kBytes, kEach = Requests::kInts * 4;
    static PerDevice<int> state;
    int ctas = 0;
    const cudaError_t e =
        resident_ctas(state, cache_attend_kernel<G, NT, C, FINE>, kBytes + kCacheMaxRequests * kEach, kBytes + 64 * kEach, &ctas);
    if (e != cudaSuccess) return e;
    return launch_pdl(cache_attend_kernel<G, NT, C, FINE>, dim3(unsigned(ctas)), dim3(kAttendThreads),
                      size_t(kBytes + a.B * kEach), s, a);
}

template <int G, int NT, int C>
cudaError_t launch_attend(const CacheAttendArgs& a, cudaStream_t s) {
    return a.dtype == 1 ? launch_attend_as<G, NT, C, true>(a, s) : launch_attend_as<G, NT, C, false>(a, s);
}

}  // namespace

cudaError_t launch_cache_attend(const CacheAttendArgs& a, cudaStream_t s) {
    if (a.total_q <= 0 || a.max_q <= 0) return cudaSuccess;
    // Columns of the matrix instruction: as few as the requests that come here can have rows.  Up to
    // four rows sit in every other column, so that each lane has one column of scores, not two
    // (64 requests, 4 rows of 128 values each: 52 us, and 55 us with all columns).
    const int64_t most = int64_t(a.max_q) * a.share;  // query rows of any request
    cudaError_t e;
    if (a.c.groups == 1)
        e = most <= 4    ? launch_attend<1, 1, 1>(a, s)
            : most <= 8  ? launch_attend<1, 1, 2>(a, s)
            : most <= 16 ? launch_attend<1, 2, 2>(a, s)
            : most <= 24 ? launch_attend<1, 3, 2>(a, s)
                         : launch_attend<1, 4, 2>(a, s);
    else
        e = most <= 4   ? launch_attend<2, 1, 1>(a, s)
            : most <= 8 ? launch_attend<2, 1, 2>(a, s)
                        : launch_attend<2, 2, 2>(a, s);
    if (e == cudaSuccess && most > few_rows(a.c.groups)) e = launch_cache_attend_rows(a, s);
    if (e != cudaSuccess || a.max_chunks <= 1) return e;
    // long memories: a row's splits are shared out among the eight warps of a CTA
    const bool wide = a.max_chunks > 16;
    const int per = wide ? 1 : 8;
    const dim3 grid(unsigned((int64_t(a.max_q) * a.q_heads + per - 1) / per), unsigned(a.B));
    auto merge = a.c.groups == 1 ? (wide ? cache_merge_kernel<1, true> : cache_merge_kernel<1, false>)
                                 : (wide ? cache_merge_kernel<2, true> : cache_merge_kernel<2, false>);
    return launch_pdl(merge, grid, dim3(256), 0, s, a);
}

}  // namespace clef
