// kda_qknorm.hip -- the norm of every head's query and key with the rotation by
// position in the same pass, and its gradients.
//
//     n = x inv,  inv = 1 / sqrt(sum(x^2) m + eps)     (m = 1, or 1 / head_dim)
//     y = scale w n,  and pairs (a, b) of y turn by the token's angle
//     backward: dy turned back, dn = scale w dy, dx = inv (dn - n m sum(dn n)),
//     dw = sum over tokens and heads of scale dy n
//
// A head is held by a few lanes, each with "slots" of two pieces of VW values: the
// first and second members of VW rotated pairs, or two pieces of the part that is
// not rotated.  So a pair never leaves its lane, every value is read once and
// written once, and HBM's rate is the bound.  Where VW does not divide a part its
// last piece is moved back over the one before: what both hold counts once.  A
// workgroup takes some tokens of q or of k; the cosines and sines of its tokens are
// formed once for all heads, angles in fp64 and reduced there, and lie in LDS, while
// the heads are read.
//
// One MI355X, bf16, replays of a graph: 65,536 tokens of 32 and 32 heads of 128, no
// rotation, 348 us (6.2 TB/s), its gradients 501 us (6.4), from fp32 ones 674 (6.4);
// 32,768 tokens of 32 and 8 heads with weights, three axes, 122 us (5.5) and 185 (5.5):
// there the wait for the table shows.  60,000 tokens of 8 and 8 heads of 77, fp32, 130 us
// (4.6).  64 tokens of 32 and 32 heads 3.4 us, a launch's own time.
#include "kda_colsum.hpp"
#include "kda_device.hpp"
#include "kda_lanes.hpp"
#include "kda_layer.hpp"

#include <algorithm>
#include <type_traits>

namespace kda {

constexpr int QK_THREADS = 256;
// Workgroups of the backward that sum a weight's gradient, of q and of k each (32,768 tokens
// of 32 and 8 heads, 384, 512, 768, 1,024: 213, 185, 186, 184 us; 16,384 of 16 and 2 heads of
// 256: 108, 92, 94, 101).
constexpr int QK_MAX_PARTIALS = 512;

enum { ROT_NONE = 0, ROT_HALVES = 1, ROT_NEIGHBOURS = 2 };

// Heads that a lane's group reads at once: more where a table of turns has to be waited
// for (32,768 tokens of 32 and 8 heads, four: 126 us, two: 139), but not in the gradients,
// whose registers they would take (with 1,024 sums a weight 194, 210 with three).
constexpr int qk_items(int rot, bool back) { return rot && !back ? 4 : 2; }

// One of q and k: its arrays, and the workgroups that take it.
struct Heads {
    const void *x;        // [T][heads][d], tokens `stride` apart
    void *y;              // forward: out, dense; backward: dx, tokens `y_stride` apart
    const void *dy;       // backward: the gradient of out, dense
    const float *weight;  // [d] or null
    float *partial;       // backward: [workgroups][d], or null
    int64_t stride, y_stride;
    int32_t heads;
    float scale;
    int32_t tile, groups;   // tokens of a tile; workgroups
    uint32_t per_head;      // 2^32 / heads, rounded up
};

struct QkShape {
    Heads of[2];
    const int32_t *positions, *pair_axis;
    const float *inv_freq;
    int32_t T, d, rot, axes;
    int32_t slots, rot_slots, lanes;   // slots of a head, those rotated, lanes of a head (a power of two)
    bool overlap;                      // pieces that share values with another
    uint32_t per_pair;                 // 2^32 / (rot / 2), rounded up (not used for one pair)
    float mean, eps;                   // m; with norm == 0 no division
    int32_t norm;
};

// Where a slot's two pieces begin, the first values of them that no other piece has
// (VW: the piece is missing), and the places of their pairs' turns.
struct Slot {
    int32_t c0, c1, f0, f1, t0, t1;
    bool rotated;
};

// Piece number p of a part of n values (at least VW) that begins at `from`: its place, and
// its first value that piece p - 1 has not.
template <int VW> __device__ __forceinline__ int32_t piece_at(int32_t from, int32_t n, int32_t p, int32_t &fresh)
{
    const int32_t at = min(VW * p, n - VW);
    fresh = min(VW * p - at, VW);
    return from + at;
}

template <int VW, int ROT> __device__ __forceinline__ Slot slot_of(const QkShape &sh, int32_t s)
{
    Slot r;
    r.rotated = ROT != ROT_NONE && s < sh.rot_slots;
    const int32_t pairs = sh.rot / 2;
    if (ROT == ROT_HALVES && r.rotated) {
        r.c0 = piece_at<VW>(0, pairs, s, r.f0);
        r.c1 = r.c0 + pairs, r.f1 = r.f0;
        r.t0 = r.t1 = r.c0;
    } else if (ROT == ROT_NEIGHBOURS && VW == 1 && r.rotated) {
        r.c0 = 2 * s, r.c1 = r.c0 + 1, r.f0 = r.f1 = 0;
        r.t0 = r.t1 = s;
    } else {   // pieces s and s + (number of slots) of the part
        const int32_t from = r.rotated ? 0 : sh.rot, n = r.rotated ? sh.rot : sh.d - sh.rot;
        const int32_t at = r.rotated ? s : s - sh.rot_slots, apart = r.rotated ? sh.rot_slots : sh.slots - sh.rot_slots;
        r.c0 = piece_at<VW>(from, n, at, r.f0);
        r.c1 = piece_at<VW>(from, n, at + apart, r.f1);
        if (VW * (at + apart) >= n) r.c1 = r.c0, r.f1 = VW;
        r.t0 = r.c0 / 2, r.t1 = r.c1 / 2;
    }
    return r;
}

// VW consecutive values, past the caches (65,536 tokens of 32 and 32 heads: 354 us, 396
// through them; 512 tokens 5.3 us either way; 1 to 512 tokens with the decode call that
// reads them 7.3 to 106 us, 0.0 to 0.2 less through them; a branch between the two costs 4 %).
template <typename T, int VW> struct QkPiece {
    typedef T raw __attribute__((ext_vector_type(VW)));
    typedef raw mem __attribute__((aligned(sizeof(T))));
    static __device__ __forceinline__ raw load(const T *p) { return __builtin_nontemporal_load(reinterpret_cast<const mem *>(p)); }
    static __device__ __forceinline__ void store(T *p, const float *v) {
        raw r;
#pragma unroll
        for (int j = 0; j < VW; ++j) r[j] = from_f<T>(v[j]);
        __builtin_nontemporal_store(r, reinterpret_cast<mem *>(p));
    }
};

// cos and sin of an angle: less whole quarters of a turn in fp64 (pi / 2 in two
// pieces), then the Taylor series of both on [-pi / 4, pi / 4], whose next terms are
// below 2^-28 there.
__device__ __forceinline__ float2 cos_sin(double angle)
{
    const double quarters = __builtin_rint(angle * 0.63661977236758134);
    double rest = __builtin_fma(-quarters, 1.5707963267948966, angle);
    rest = __builtin_fma(-quarters, 6.123233995736766e-17, rest);
    const float r = (float)rest, z = r * r;
    float sn = __builtin_fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
    sn = __builtin_fmaf(z, sn, 1.f / 120.f);
    sn = __builtin_fmaf(z, sn, -1.f / 6.f);
    sn = __builtin_fmaf(r * z, sn, r);
    float cs = __builtin_fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
    cs = __builtin_fmaf(z, cs, -1.f / 720.f);
    cs = __builtin_fmaf(z, cs, 1.f / 24.f);
    cs = __builtin_fmaf(z, cs, -0.5f);
    cs = __builtin_fmaf(z, cs, 1.f);
    const int q = (int)(int64_t)quarters;   // (its last two bits; an angle that is no number gives NaN above)
    const float a = q & 1 ? sn : cs, b = q & 1 ? cs : sn;
    return float2{(q + 1) & 2 ? -a : a, q & 2 ? -b : b};
}

// cos and sin of tokens [t0, t0 + count) into table[token][pair]
__device__ __forceinline__ void turn_table(const QkShape &sh, int64_t t0, int32_t count, float2 *table)
{
    const int32_t pairs = sh.rot / 2;
    for (int32_t i = threadIdx.x; i < count * pairs; i += QK_THREADS) {
        const int32_t t = pairs == 1 ? i : (int32_t)__umulhi((uint32_t)i, sh.per_pair), j = i - t * pairs;   // i / pairs
        const int32_t axis = sh.pair_axis ? min(max(sh.pair_axis[j], 0), sh.axes - 1) : 0;
        table[i] = cos_sin((double)sh.positions[(int64_t)axis * sh.T + t0 + t] * (double)sh.inv_freq[j]);
    }
}

// Turns a slot's pairs, by their angles or (back) against them.
template <int VW, int ROT, bool AGAINST> __device__ __forceinline__ void turn(float *v, const Slot &sl, const float2 *turns)
{
    const auto pair = [](float &a, float &b, float2 t) {
        const float sn = AGAINST ? -t.y : t.y, a1 = a * t.x - b * sn;
        b = b * t.x + a * sn;
        a = a1;
    };
    if (ROT == ROT_HALVES || VW == 1) {
#pragma unroll
        for (int j = 0; j < VW; ++j) pair(v[j], v[VW + j], turns[sl.t0 + j]);
    } else {
#pragma unroll
        for (int j = 0; j < VW / 2; ++j) pair(v[2 * j], v[2 * j + 1], turns[sl.t0 + j]);
#pragma unroll
        for (int j = 0; j < VW / 2; ++j) pair(v[VW + 2 * j], v[VW + 2 * j + 1], turns[sl.t1 + j]);
    }
}

// the sums over a head's lanes
template <int M> __device__ __forceinline__ void head_sums(float (&s)[M], int32_t lanes)
{
#pragma unroll
    for (int m = 0; m < M; ++m) {
        if (lanes >= 2) s[m] += dpp<DPP_XOR1>(s[m]);
        if (lanes >= 4) s[m] += dpp<DPP_XOR2>(s[m]);
        if (lanes >= 8) s[m] += dpp<DPP_HALF_MIRROR>(s[m]);
        if (lanes >= 16) s[m] += dpp<DPP_MIRROR>(s[m]);
        if (lanes >= 32) s[m] = add_xor16(s[m]);
        if (lanes >= 64) s[m] = add_xor32(s[m]);
    }
}

// The forward and the gradients walk the same items: (token, head) number
// `item` of a workgroup's tile of tokens.  C slots a lane.
template <typename T, typename G, int VW, int C, int ROT, bool BACK>
__global__ __launch_bounds__(QK_THREADS, 3) void kda_qknorm_kernel(QkShape sh)
{
    typedef QkPiece<T, VW> P;
    typedef QkPiece<G, VW> PG;
    constexpr int ITEMS = qk_items(ROT, BACK);
    extern __shared__ float2 table[];
    const bool second = (int32_t)blockIdx.x >= sh.of[0].groups;
    const Heads hd = second ? sh.of[1] : sh.of[0];
    const int32_t group = (int32_t)blockIdx.x - (second ? sh.of[0].groups : 0);
    const int32_t lane = threadIdx.x & (sh.lanes - 1), per = QK_THREADS / sh.lanes, g0 = threadIdx.x / sh.lanes;
    const T *const xs = (const T *)hd.x;
    const G *const dys = (const G *)hd.dy;
    T *const ys = (T *)hd.y;
    const int32_t pairs = sh.rot / 2;
    float dw[C][2 * VW] = {}, w[C][2 * VW];
    Slot sl[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int32_t s = lane + c * sh.lanes;
        sl[c] = slot_of<VW, ROT>(sh, min(s, sh.slots - 1));
        if (s >= sh.slots) sl[c].f0 = sl[c].f1 = VW, sl[c].rotated = false;
#pragma unroll
        for (int j = 0; j < 2 * VW; ++j) w[c][j] = hd.weight ? hd.weight[(j < VW ? sl[c].c0 : sl[c].c1 - VW) + j] : 1.f;
    }

    struct Batch {
        typename P::raw x[ITEMS][C][2];
        typename PG::raw dy[ITEMS][C][2];
        int32_t token[ITEMS];
        int64_t at[ITEMS];
        bool live[ITEMS];
    };
    for (int64_t t0 = (int64_t)group * hd.tile; t0 < sh.T; t0 += (int64_t)hd.groups * hd.tile) {
        const int32_t count = (int32_t)min((int64_t)hd.tile, sh.T - t0), items = count * hd.heads;
        // reads the heads of items i0, i0 + per, ...
        const auto fetch = [&](int32_t i0) {
            Batch in;
#pragma unroll
            for (int u = 0; u < ITEMS; ++u) {
                const int32_t item = i0 + u * per;
                in.live[u] = item < items;
                // item / heads (items are below 2^12 where a tile has several tokens)
                in.token[u] = !in.live[u] || hd.tile == 1 ? 0 : hd.heads == 1 ? item : (int32_t)__umulhi((uint32_t)item, hd.per_head);
                const int32_t head = in.live[u] ? item - in.token[u] * hd.heads : 0;
                in.at[u] = ((t0 + in.token[u]) * hd.heads + head) * sh.d;
                const T *row = xs + (t0 + in.token[u]) * hd.stride + (int64_t)head * sh.d;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    in.x[u][c][0] = in.x[u][c][1] = typename P::raw{};
                    if (BACK) in.dy[u][c][0] = in.dy[u][c][1] = typename PG::raw{};
                    if (sl[c].f0 < VW) {
                        in.x[u][c][0] = P::load(row + sl[c].c0);
                        if (BACK) in.dy[u][c][0] = PG::load(dys + in.at[u] + sl[c].c0);
                    }
                    if (sl[c].f1 < VW) {
                        in.x[u][c][1] = P::load(row + sl[c].c1);
                        if (BACK) in.dy[u][c][1] = PG::load(dys + in.at[u] + sl[c].c1);
                    }
                }
            }
            return in;
        };
        Batch in = fetch(g0);
        if (ROT) {   // the table while they arrive
            turn_table(sh, t0, count, table);
            __syncthreads();
        }
        for (int32_t i0 = g0; i0 - g0 < items; i0 += per * ITEMS) {
            if (i0 != g0) in = fetch(i0);
#pragma unroll
            for (int u = 0; u < ITEMS; ++u) {
                float v[C][2 * VW], e[C][2 * VW];
                float sum[BACK ? 2 : 1] = {};
#pragma unroll
                for (int c = 0; c < C; ++c) {
#pragma unroll
                    for (int j = 0; j < VW; ++j) v[c][j] = to_f(in.x[u][c][0][j]), v[c][VW + j] = to_f(in.x[u][c][1][j]);
                    if (BACK) {
#pragma unroll
                        for (int j = 0; j < VW; ++j) {
                            e[c][j] = to_f(in.dy[u][c][0][j]) * hd.scale;
                            e[c][VW + j] = to_f(in.dy[u][c][1][j]) * hd.scale;
                        }
                        if (ROT && sl[c].rotated) turn<VW, ROT, true>(e[c], sl[c], table + in.token[u] * pairs);
                    }
                    // (e: the gradient of w n)
                    const auto add = [&](int j) {
                        sum[0] += v[c][j] * v[c][j];
                        if (BACK) sum[BACK ? 1 : 0] += e[c][j] * w[c][j] * v[c][j];
                    };
                    if (sh.overlap) {
#pragma unroll
                        for (int j = 0; j < 2 * VW; ++j)
                            if (j < VW ? j >= sl[c].f0 : j - VW >= sl[c].f1) add(j);
                    } else {
#pragma unroll
                        for (int j = 0; j < 2 * VW; ++j) add(j);
                    }
                }
                head_sums(sum, sh.lanes);
                const float inv = sh.norm ? 1.f / sqrtf(sum[0] * sh.mean + sh.eps) : 1.f;
                const float along = BACK && sh.norm ? sum[BACK ? 1 : 0] * inv * sh.mean * inv : 0.f;   // of x, not of n
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    if (!in.live[u]) continue;
                    T *row;
                    if (!BACK) {
#pragma unroll
                        for (int j = 0; j < 2 * VW; ++j) v[c][j] *= inv * hd.scale, v[c][j] *= w[c][j];
                        if (ROT && sl[c].rotated) turn<VW, ROT, false>(v[c], sl[c], table + in.token[u] * pairs);
                        row = ys + in.at[u];
                    } else {
#pragma unroll
                        for (int j = 0; j < 2 * VW; ++j) {
                            dw[c][j] += e[c][j] * (v[c][j] * inv);
                            // (a selection: without a norm an infinite x has no part in its gradient)
                            v[c][j] = inv * (e[c][j] * w[c][j] - (sh.norm ? along * v[c][j] : 0.f));
                        }
                        // (the same token and head, at dx's own stride)
                        row = ys + (t0 + in.token[u]) * hd.y_stride + (in.at[u] - (t0 + in.token[u]) * hd.heads * sh.d);
                    }
                    if (sl[c].f0 < VW) P::store(row + sl[c].c0, v[c]);
                    if (sl[c].f1 < VW) P::store(row + sl[c].c1, v[c] + VW);
                }
            }
        }
        if (ROT) __syncthreads();   // the table is done with
    }
    if (!BACK || !hd.partial) return;
    // the sums of a slot's values over the groups, in order: a value a thread (32,768 tokens of
    // 32 and 8 heads 185 us, 8 tokens 8.2; by the first group alone 190 and 14.5)
    float *fold = reinterpret_cast<float *>(table);
    const int32_t pitch = QK_THREADS + sh.lanes;   // (values of a wave on different banks)
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 2 * VW; ++j) fold[(c * 2 * VW + j) * pitch + threadIdx.x] = dw[c][j];
    __syncthreads();
    for (int32_t i = threadIdx.x; i < sh.lanes * C * 2 * VW; i += QK_THREADS) {
        const int32_t l = i & (sh.lanes - 1), value = i / sh.lanes, j = value % (2 * VW), s = l + value / (2 * VW) * sh.lanes;
        if (s >= sh.slots) continue;
        const Slot of = slot_of<VW, ROT>(sh, s);
        if (j < VW ? j < of.f0 : j - VW < of.f1) continue;
        const float *part = fold + value * pitch + l;
        float sum = 0.f;
#pragma unroll 4
        for (int32_t g = 0; g < per; ++g) sum += part[g * sh.lanes];
        hd.partial[(int64_t)group * sh.d + (j < VW ? of.c0 : of.c1 - VW) + j] = sum;
    }
}

// dq_weight and dk_weight: the sums over the workgroups' parts
__global__ __launch_bounds__(COLSUM_THREADS) void kda_qknorm_weights_kernel(const float *part0, int32_t n0, float *dst0,
                                                                            const float *part1, int32_t n1, float *dst1,
                                                                            int32_t d)
{
    const bool second = blockIdx.y == 1;
    const float *part = second ? part1 : part0;
    float *dst = second ? dst1 : dst0;
    if (!dst) return;
    const int64_t c = (int64_t)blockIdx.x * COLSUM_COLS + threadIdx.x % COLSUM_COLS;
    const float s = column_sum(part, second ? n1 : n0, d, c);
    if (threadIdx.x < COLSUM_COLS && c < d) dst[c] = s;
}

// ---------------------------------------------------------------- host
// The slots of a head with pieces of `w` values: those rotated, and all.
inline int32_t ceil_div(int32_t a, int32_t b) { return (a + b - 1) / b; }
inline int32_t rotated_slots(const QkShape &sh, int mode, int w)
{
    return mode == ROT_NONE ? 0 : mode == ROT_HALVES ? ceil_div(sh.rot / 2, w) : w == 1 ? sh.rot / 2 : ceil_div(ceil_div(sh.rot, w), 2);
}
inline int32_t all_slots(const QkShape &sh, int mode, int w)
{
    return rotated_slots(sh, mode, w) + ceil_div(ceil_div(sh.d - sh.rot, w), 2);
}

// The slots and lanes of a head, and the tiles: as many tokens as a workgroup takes
// heads at once, `items` a lane's group.
template <int VW, int C> void lay_out(QkShape &sh, int mode, int items)
{
    sh.rot_slots = rotated_slots(sh, mode, VW);
    sh.slots = all_slots(sh, mode, VW);
    sh.overlap = (mode == ROT_HALVES ? sh.rot / 2 : sh.rot) % VW != 0 || (sh.d - sh.rot) % VW != 0;
    sh.per_pair = sh.rot > 2 ? (uint32_t)((((uint64_t)1 << 32) + sh.rot / 2 - 1) / (sh.rot / 2)) : 0;
    sh.lanes = 1;
    while (sh.lanes * C < sh.slots) sh.lanes *= 2;
    const int32_t at_once = QK_THREADS / sh.lanes * items;
    for (Heads &h : sh.of) {
        const auto tokens_of = [&](int32_t n) { return h.heads ? (n + h.heads - 1) / h.heads : 1; };
        // a round of heads at least; more while 256 workgroups are left (64 tokens of 32 and 8
        // heads with three axes, 2 and 8 tokens of k: 5.5 and 7.5 us)
        h.tile = std::max(tokens_of(QK_THREADS / sh.lanes), std::min(tokens_of(at_once), sh.T / 256));
        // (a table of 32 KB at most: five workgroups a CU)
        if (sh.rot) h.tile = std::min(h.tile, std::max(1, 4096 / (sh.rot / 2)));
        h.per_head = h.heads > 1 ? (uint32_t)((((uint64_t)1 << 32) + h.heads - 1) / h.heads) : 0;
        h.groups = h.heads ? (int32_t)(((int64_t)sh.T + h.tile - 1) / h.tile) : 0;
        // sums of a weight's gradient: few workgroups, which take several tiles
        if (h.partial) h.groups = std::min(h.groups, QK_MAX_PARTIALS);
    }
}

template <typename T, typename G, int VW, int C, int ROT, bool BACK> hipError_t run_qknorm(QkShape sh, hipStream_t s)
{
    const int32_t groups = sh.of[0].groups + sh.of[1].groups;
    if (groups == 0) return hipSuccess;
    size_t lds = 0;
    if (ROT)
        for (const Heads &h : sh.of) lds = std::max(lds, sizeof(float2) * h.tile * (size_t)(sh.rot / 2));
    if (BACK && (sh.of[0].partial || sh.of[1].partial)) lds = std::max(lds, sizeof(float) * (QK_THREADS + sh.lanes) * C * 2 * VW);
    hipLaunchKernelGGL((kda_qknorm_kernel<T, G, VW, C, ROT, BACK>), dim3((unsigned)groups), dim3(QK_THREADS), lds, s, sh);
    return hipGetLastError();
}

// Calls f with the width of a piece and the slots of a lane: the widest piece, of
// 16 bytes at most, that no part of a head is shorter than (60,000 tokens of 8 and 8
// heads of 77, fp32: 130 us, with pieces of the one value that divides 77 231).
template <typename T, typename Fn> auto with_width(const QkShape &sh, int mode, Fn f)
{
    const auto fits = [&](int w) {
        return (sh.rot == 0 || (mode == ROT_HALVES ? sh.rot / 2 : sh.rot) >= w) && (sh.d == sh.rot || sh.d - sh.rot >= w);
    };
    if constexpr (sizeof(T) == 2) {
        if (fits(8)) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
    } else {
        if (fits(4) && all_slots(sh, mode, 4) <= 64) return f(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
    }
    if (fits(4)) return f(std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
    if (fits(2)) return f(std::integral_constant<int, 2>(), std::integral_constant<int, 4>());
    return f(std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
}

template <typename T, typename G, bool BACK> hipError_t qknorm(QkShape sh, int mode, hipStream_t s)
{
    return with_width<T>(sh, mode, [&](auto w, auto c) {
        lay_out<w(), c()>(sh, mode, qk_items(mode, BACK));
        return mode == ROT_NONE     ? run_qknorm<T, G, w(), c(), ROT_NONE, BACK>(sh, s)
               : mode == ROT_HALVES ? run_qknorm<T, G, w(), c(), ROT_HALVES, BACK>(sh, s)
                                    : run_qknorm<T, G, w(), c(), ROT_NEIGHBOURS, BACK>(sh, s);
    });
}

}  // namespace kda

using namespace kda;

static int qk_mode(int32_t rot, bool interleaved) { return rot == 0 ? ROT_NONE : interleaved ? ROT_NEIGHBOURS : ROT_HALVES; }

static QkShape qk_shape(const KdaQkNorm &a)
{
    QkShape sh{};
    sh.of[0] = {a.q, nullptr, nullptr, a.q_weight, nullptr, a.q_stride, 0, a.q_heads, a.q_scale, 0, 0, 0};
    sh.of[1] = {a.k, nullptr, nullptr, a.k_weight, nullptr, a.k_stride, 0, a.k_heads, 1.f, 0, 0, 0};
    sh.positions = a.positions, sh.pair_axis = a.pair_axis, sh.inv_freq = a.inv_freq;
    sh.T = a.tokens, sh.d = a.dim, sh.rot = a.rot, sh.axes = a.axes;
    sh.mean = a.norm == 2 ? 1.f / a.dim : 1.f, sh.eps = a.eps, sh.norm = a.norm;
    return sh;
}

hipError_t kda_launch_qknorm(bool bf16, const KdaQkNorm &a, void *q_out, void *k_out, hipStream_t s)
{
    QkShape sh = qk_shape(a);
    sh.of[0].y = q_out, sh.of[1].y = k_out;
    const int mode = qk_mode(a.rot, a.interleaved);
    return bf16 ? qknorm<bf16_t, bf16_t, false>(sh, mode, s) : qknorm<float, float, false>(sh, mode, s);
}

size_t kda_qknorm_bwd_ws_bytes(int32_t d) { return sizeof(float) * 2 * QK_MAX_PARTIALS * (size_t)d; }

hipError_t kda_launch_qknorm_backward(bool bf16, bool grad_bf16, const KdaQkNorm &a, const void *dq_out, const void *dk_out,
                                      int64_t dq_stride, int64_t dk_stride, void *dq, void *dk, float *dq_weight,
                                      float *dk_weight, void *ws, hipStream_t s)
{
    QkShape sh = qk_shape(a);
    float *const part0 = (float *)ws, *const part1 = part0 + (size_t)QK_MAX_PARTIALS * a.dim;
    sh.of[0].y = dq, sh.of[0].y_stride = dq_stride, sh.of[0].dy = dq_out, sh.of[0].partial = dq_weight ? part0 : nullptr;
    sh.of[1].y = dk, sh.of[1].y_stride = dk_stride, sh.of[1].dy = dk_out, sh.of[1].partial = dk_weight ? part1 : nullptr;
    const int mode = qk_mode(a.rot, a.interleaved);
    hipError_t e = hipSuccess;
    int32_t groups[2] = {0, 0};
    const auto run = [&](auto t, auto g) {
        typedef decltype(t) T;
        typedef decltype(g) G;
        with_width<T>(sh, mode, [&](auto w, auto c) {
            lay_out<w(), c()>(sh, mode, qk_items(mode, true));
            return 0;
        });
        groups[0] = sh.of[0].groups, groups[1] = sh.of[1].groups;
        return qknorm<T, G, true>(sh, mode, s);
    };
    e = !bf16 ? run(float(), float()) : grad_bf16 ? run(bf16_t(), bf16_t()) : run(bf16_t(), float());
    if (e != hipSuccess || (!dq_weight && !dk_weight)) return e;
    hipLaunchKernelGGL(kda_qknorm_weights_kernel, dim3((unsigned)((a.dim + COLSUM_COLS - 1) / COLSUM_COLS), 2),
                       dim3(COLSUM_THREADS), 0, s, (const float *)part0, groups[0], dq_weight, (const float *)part1, groups[1],
                       dk_weight, a.dim);
    return hipGetLastError();
}

bool kda_qknorm_fits(bool bf16, const KdaQkNorm &a, bool back)
{
    QkShape sh = qk_shape(a);
    const int mode = qk_mode(a.rot, a.interleaved);
    const auto groups = [&](auto w, auto c) {
        lay_out<w(), c()>(sh, mode, qk_items(mode, back));
        return (int64_t)sh.of[0].groups + sh.of[1].groups;
    };
    return kda_grid_ok(bf16 ? with_width<bf16_t>(sh, mode, groups) : with_width<float>(sh, mode, groups), QK_THREADS);
}
