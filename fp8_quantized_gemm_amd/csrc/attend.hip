// Attention over the paged FP8 cache for few query rows (see paged.hpp).
#include "join.hpp"

namespace fp8q {
namespace {

constexpr int kWaves = 4, kThreads = kWaves * 64;
constexpr int kPolicy = CP_DEFAULT;
constexpr int kRows = 16;                 // query rows of a unit: (token, head of the group) pairs
constexpr int kKeys = 64;                 // keys of a tile
// Two workgroups on each of 256 CUs, one from 192 channels on (registers).
constexpr int groups_for(int dp) { return dp <= 128 ? 512 : 256; }
// Waves of a workgroup: eight where it takes a whole unit and the registers allow.
constexpr int waves_for(int dp, bool shared) { return shared || dp > 128 ? 4 : 8; }
constexpr int kMinShare = 3;              // what a wave takes at least

// The work is a list of units (sequence, key/value head, row tile), each a run of
// key tiles with one place before them for what a unit costs by itself; wave i
// of the grid takes the places [i * share, (i + 1) * share) of the whole list.
// That evens out any mixture of lengths, and is computed from the batch's arrays
// by every workgroup, so the host needs no lengths and a graph can be replayed
// with others.  A wave stores the units that it has whole; the pieces of the
// others are joined in LDS, and those of units that several workgroups have by
// attend_join_kernel.
struct SeqWork {
    PagedSeq q;
    int tile0, tiles;                     // key tiles that some row of the sequence sees
    int row_tiles;
    __device__ __forceinline__ int64_t places(int Hk) const { return (int64_t)row_tiles * Hk * (tiles + 1); }
};

__device__ __forceinline__ SeqWork seq_work(const AttendArgs& a, int b)
{
    SeqWork w;
    w.q = paged_seq(a.batch, b, a.P);
    const KeyRange first = key_range(a, w.q, 0), last = key_range(a, w.q, w.q.n - 1);
    w.tile0 = first.lo / kKeys;
    w.tiles = max((last.hi + kKeys - 1) / kKeys - w.tile0, 1);
    w.row_tiles = (w.q.n * a.group + kRows - 1) / kRows;
    return w;
}

struct ScanLds {
    int64_t sums[kWaves];
    int64_t before[kWaves];
    int seq[kWaves];
};

__device__ __forceinline__ int64_t share_of(int64_t total, int waves)
{
    const int64_t s = (total + waves - 1) / waves;
    return s > kMinShare ? s : kMinShare;
}

// Places of all sequences, and for the first place of each of the workgroup's waves the
// sequence that holds it and the places before that sequence.  Every thread sums a run of
// sequences.
__device__ __forceinline__ int64_t scan_sequences(const AttendArgs& a, ScanLds& lds)
{
    const int B = a.batch.B, per = (B + kThreads - 1) / kThreads, lane = threadIdx.x & 63;
    const int b0 = min((int)threadIdx.x * per, B), b1 = min(b0 + per, B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += seq_work(a, b).places(a.Hk);
    int64_t sum = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t up = __shfl_up(sum, off);
        if (lane >= off) sum += up;
    }
    if (lane == 63) lds.sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    int64_t total = 0, before = sum - mine;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < (int)(threadIdx.x >> 6)) before += lds.sums[w];
        total += lds.sums[w];
    }
    const int64_t share = share_of(total, gridDim.x * kWaves);
    for (int w = 0; w < kWaves; ++w) {
        const int64_t at = ((int64_t)blockIdx.x * kWaves + w) * share;
        if (at < before || at >= before + mine) continue;
        int64_t from = before;
        for (int b = b0; b < b1; ++b) {
            const int64_t n = seq_work(a, b).places(a.Hk);
            if (at < from + n) {
                lds.seq[w] = b;
                lds.before[w] = from;
                break;
            }
            from += n;
        }
    }
    __syncthreads();
    return total;
}

// The scratch: for each workgroup the unit that it begins and another one ends (parts = 0:
// none), then its two partial results, of a unit that it goes on with and of one that it
// begins: kRows rows of maximum, denominator and, from the fifth float on, DP sums.
template <int DP>
__host__ __device__ __forceinline__ float* part_of(float* work, int groups, int64_t group, bool begins)
{
    return work + groups * (int)(sizeof(Unit) / 4) + (group * 2 + (begins ? 1 : 0)) * (kRows * (DP + 4));
}

// A key tile as a wave holds it: lane (r, g) has 16 channels for each 64 of the keys
// 16 (r / 4) + 4 i + r % 4, i < 4, and the 16 keys from 16 g on of the channels 16 d + r.
template <int DP>
struct KvTile {
    v4i k[4][DP / 64], v[DP / 16];
};

// What a wave knows of the pages of the next tiles: lane i of the page with the i-th of 64 tiles where
// a page holds whole tiles (WIDE), else of the i-th of 64 groups of 16 keys.  Looked up together, so
// that no tile waits for its page's id or scales.
struct Pages {
    int page;                             // 0 where there is none
    PageScales sc;
    uint64_t valid;
};
template <bool WIDE>
constexpr int kLookUp = WIDE ? 64 : 16;   // tiles of a look-up
template <bool WIDE>
__device__ __forceinline__ Pages look_up(const AttendArgs& a, int b, int len, int key0, int h)
{
    const int key = key0 + (int)(threadIdx.x & 63) * (WIDE ? kKeys : 16);
    const PageRef p = page_ref(a, b, len, key);
    return Pages{(int)p.page, page_scales(a, p.page, h), __ballot(p.valid)};
}
// What a lane needs of the i-th tile of a look-up: the pages of the keys and of the values that it
// loads, the scales of its terms.
struct TilePages {
    int k, v, k_inside, v_inside;
    PageScales sc;
    bool valid;
};
template <bool WIDE>
__device__ __forceinline__ TilePages tile_pages(const AttendArgs& a, const Pages& p, int i, int key0, int r, int g)
{
    if constexpr (WIDE) {
        const auto lane_i = [&](float v) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i)); };
        const int page = __builtin_amdgcn_readlane(p.page, i), inside = key0 & (a.P - 1);
        return TilePages{page, page, inside, inside,
                         PageScales{lane_i(p.sc.key), lane_i(p.sc.log_value), lane_i(p.sc.inverse_value)},
                         (p.valid >> i & 1) != 0};
    } else {
        const int ik = 4 * i + (r >> 2), iv = 4 * i + g;
        return TilePages{__shfl(p.page, ik), __shfl(p.page, iv), (key0 + 16 * (r >> 2)) & (a.P - 1),
                         (key0 + 16 * g) & (a.P - 1),
                         PageScales{__shfl(p.sc.key, iv), __shfl(p.sc.log_value, iv), __shfl(p.sc.inverse_value, iv)},
                         (p.valid >> iv & 1) != 0};
    }
}

template <int DP, bool WIDE>
__device__ __forceinline__ void load_keys(const AttendArgs& a, KvTile<DP>& t, const TilePages& p, int h,
                                          int r, int g)
{
    constexpr int NC = DP / 64;
    const int64_t page_bytes = (int64_t)a.P * a.D, pool_stride = a.Hk * page_bytes;
    if constexpr (WIDE) {
        // buffer loads: one 32-bit offset a lane, the rest scalar; channels past D are sent out of
        // the buffer's range and read as 0
        const rsrc_t rk = make_rsrc(a.k_pages + p.k * pool_stride + h * page_bytes + p.k_inside * a.D,
                                    (uint32_t)(kKeys * a.D));
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = 64 * c + 16 * g;
                const uint32_t at = (uint32_t)((16 * (r >> 2) + (r & 3)) * a.D + d);
                t.k[i][c] = __builtin_amdgcn_raw_buffer_load_b128(rk, d < a.D ? at : kOOB, uniform(4 * i * a.D),
                                                                  kPolicy);
            }
    } else {
        const uint8_t* kt = a.k_pages + p.k * pool_stride + h * page_bytes +
                            (int64_t)(p.k_inside + (r & 3)) * a.D;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = 64 * c + 16 * g;
                t.k[i][c] = v4i{0, 0, 0, 0};
                if (d < a.D) t.k[i][c] = *reinterpret_cast<const v4i*>(kt + 4 * i * a.D + d);
            }
    }
}

template <int DP, bool WIDE>
__device__ __forceinline__ void load_values(const AttendArgs& a, KvTile<DP>& t, const TilePages& p, int h,
                                            int r, int g)
{
    constexpr int ND = DP / 16;
    const int64_t page_bytes = (int64_t)a.P * a.D, pool_stride = a.Hk * page_bytes;
    if constexpr (WIDE) {
        const rsrc_t rv = make_rsrc(a.v_pages + p.v * pool_stride + h * page_bytes + p.v_inside,
                                    (uint32_t)(page_bytes - p.v_inside));
#pragma unroll
        for (int d = 0; d < ND; ++d)
            t.v[d] = __builtin_amdgcn_raw_buffer_load_b128(rv, (uint32_t)(r * a.P + 16 * g),
                                                           uniform(16 * d * a.P), kPolicy);
    } else {
        const uint8_t* vt = a.v_pages + p.v * pool_stride + h * page_bytes + p.v_inside;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            t.v[d] = v4i{0, 0, 0, 0};
            if (16 * d < a.D) t.v[d] = *reinterpret_cast<const v4i*>(vt + (int64_t)(16 * d + r) * a.P);
        }
    }
}

// What a wave has of 16 query rows: lane (r, g) the sums of row r's channels 16 d + 4 g ..,
// the reference, and its own keys' share of the denominator.
template <int DP>
struct Rows {
    v4i q[DP / 64][2];
    v4f acc[DP / 16];
    float m, l;
};

// A tile's terms; keys_read is called when its keys are no longer needed.
template <int DT, int DP, class F>
__device__ __forceinline__ void add_tile(Rows<DP>& x, KvTile<DP>& t, const PageScales& sc, const KeyRange& see,
                                         bool whole, bool valid, int key0, int g, F keys_read)
{
    constexpr int NC = DP / 64, ND = DP / 16;
    v4f s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            s[i] = Half<DT>::mfma(Half<DT>::widen(t.k[i][c][0], t.k[i][c][1]), x.q[c][0], s[i]);
            s[i] = Half<DT>::mfma(Half<DT>::widen(t.k[i][c][2], t.k[i][c][3]), x.q[c][1], s[i]);
        }
    }
    keys_read();
    if (!whole) mask_tile<ND>(s, x.acc, t.v, see, key0, g, valid);

    float top = s[0][0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i >> 2][i & 3]);
    top = __builtin_fmaf(top, sc.key, sc.log_value);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    if (__any(top > x.m + kSlack)) {
        const float m1 = fmaxf(x.m, top);
        const float alpha = m1 == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(x.m - m1);
        x.l *= alpha;
#pragma unroll
        for (int d = 0; d < ND; ++d) x.acc[d] *= alpha;
        x.m = m1;
    }
    const float offset = sc.log_value - ((x.m == -__builtin_inff() ? 0.0f : x.m) - kShift);
    float sum = 0.0f;
    v8h p[2];
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const v2f v = {__builtin_amdgcn_exp2f(__builtin_fmaf(s[i >> 2][i & 3], sc.key, offset)),
                       __builtin_amdgcn_exp2f(__builtin_fmaf(s[i >> 2][(i & 3) + 1], sc.key, offset))};
        sum += v[0];
        sum += v[1];
        const v2h w = __builtin_convertvector(v, v2h);
        p[i >> 3][i & 7] = w[0];
        p[i >> 3][(i & 7) + 1] = w[1];
    }
    x.l = __builtin_fmaf(sum, sc.inverse_value, x.l);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        x.acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(Half<DT_FP16>::widen(t.v[d][0], t.v[d][1]), p[0],
                                                          x.acc[d], 0, 0, 0);
        x.acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(Half<DT_FP16>::widen(t.v[d][2], t.v[d][3]), p[1],
                                                          x.acc[d], 0, 0, 0);
    }
}

// A run of tiles [t0, t1) of a unit (key/value head h, rows from row0 on) by one wave.
struct Run {
    int h, row0, rows, t0, t1;
};
template <int DT, int DP, bool WIDE>
__device__ __forceinline__ void attend_run(const AttendArgs& a, int b, const SeqWork& w, const Run& u, Rows<DP>& x,
                                           int& token, int& head)
{
    constexpr int NC = DP / 64, ND = DP / 16;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, h = u.h;
    // this lane's query row and the keys it sees
    const int my_row = u.row0 + r;
    token = my_row / a.group;
    head = h * a.group + (my_row - token * a.group);
    KeyRange see = key_range(a, w.q, token);
    if (r >= u.rows) see.lo = see.hi = 0;
    const KeyRange first = key_range(a, w.q, uniform(token)),
                   last = key_range(a, w.q, __builtin_amdgcn_readlane(token, u.rows - 1));
    const auto key_of = [&](int t) { return (w.tile0 + t) * kKeys; };
    Pages known = look_up<WIDE>(a, b, w.q.len, key_of(u.t0), h);
    {
        const uint16_t* src = a.q + (int64_t)(w.q.row + token) * a.q_stride + (int64_t)head * a.D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = 64 * c + 16 * g;
            const bool have = r < u.rows && d < a.D;
            const v4i zero = {0, 0, 0, 0};
            x.q[c][0] = have ? *reinterpret_cast<const v4i*>(src + d) ^ a.q_flip : zero;
            x.q[c][1] = have ? *reinterpret_cast<const v4i*>(src + d + 8) ^ a.q_flip : zero;
        }
    }
#pragma unroll
    for (int d = 0; d < ND; ++d) x.acc[d] = v4f{0.f, 0.f, 0.f, 0.f};
    x.m = -__builtin_inff();
    x.l = 0.0f;

    // the next tile's keys are asked for when this tile's have been read, its values likewise
    KvTile<DP> tile;
    TilePages pages = tile_pages<WIDE>(a, known, 0, key_of(u.t0), r, g);
    load_keys<DP, WIDE>(a, tile, pages, h, r, g);
    load_values<DP, WIDE>(a, tile, pages, h, r, g);
    for (int t = u.t0; t < u.t1; ++t) {
        const int key0 = key_of(t), next = (t + 1 - u.t0) % kLookUp<WIDE>;
        const bool more = t + 1 < u.t1;
        const bool whole = first.lo <= key0 && last.lo <= key0 && first.hi >= key0 + kKeys &&
                           last.hi >= key0 + kKeys && __all(pages.valid);
        const PageScales sc = pages.sc;
        const bool valid = pages.valid;
        add_tile<DT, DP>(x, tile, sc, see, whole, valid, key0, g, [&] {
            if (!more) return;
            if (next == 0) known = look_up<WIDE>(a, b, w.q.len, key0 + kKeys, h);
            pages = tile_pages<WIDE>(a, known, next, key0 + kKeys, r, g);
            load_keys<DP, WIDE>(a, tile, pages, h, r, g);
        });
        if (more) load_values<DP, WIDE>(a, tile, pages, h, r, g);
    }
    x.l += __shfl_xor(x.l, 16);                             // the lane groups had keys of their own
    x.l += __shfl_xor(x.l, 32);
}

// SHARED: the grid's waves share the list of all units' tiles.  Else a workgroup takes one unit,
// its waves equal runs of the tiles.
template <int DT, int DP, bool WIDE, bool SHARED>
__global__ void __launch_bounds__(waves_for(DP, SHARED) * 64, DP <= 128 ? 2 : 1)
    attend_rows_kernel(const AttendArgs a)
{
    constexpr int kWaves = waves_for(DP, SHARED), kThreads = kWaves * 64, kPieces = SHARED ? 2 * kWaves : kWaves;
    constexpr int ND = DP / 16;
    constexpr int RS = DP + 4;                              // floats of a row in LDS
    __shared__ Unit piece[kPieces];
    __shared__ float stat[kPieces][kRows][2];
    __shared__ __attribute__((aligned(16))) float sums[kPieces][kRows * RS];

    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const auto keep = [&](const SeqWork& w, const Run& u, const Rows<DP>& x, int slot, int64_t unit_at, int parts) {
        if (g == 0) { stat[slot][r][0] = x.m; stat[slot][r][1] = x.l; }
#pragma unroll
        for (int d = 0; d < ND; ++d) *reinterpret_cast<v4f*>(&sums[slot][r * RS + 16 * d + 4 * g]) = x.acc[d];
        if (lane == 0)
            piece[slot] = Unit{unit_at, parts, u.t0 == 0, u.t1 == w.tiles, w.q.row, u.h, u.row0, u.rows, 0};
    };
    const auto store = [&](const SeqWork& w, const Run& u, const Rows<DP>& x, int token, int head) {
        const Joined j{x.m, x.m == -__builtin_inff() ? 0.0f : x.m, x.l};
        if (r < u.rows)
#pragma unroll
            for (int d = 0; d < ND; ++d)
                if (16 * d < a.D) store_row<DT>(a, w.q.row + token, head, 16 * d + 4 * g, x.acc[d], j);
    };
    Rows<DP> x;
    int token, head;
    if constexpr (SHARED) {
        __shared__ ScanLds scan;
        const int64_t total = uniform(scan_sequences(a, scan)), share = share_of(total, gridDim.x * kWaves);
        int64_t at = ((int64_t)blockIdx.x * kWaves + wave) * share, seq_at = 0;
        const int64_t end = at + share < total ? at + share : total;
        int b = 0;
        if (at < end) {
            b = uniform(scan.seq[wave]);
            seq_at = uniform(scan.before[wave]);
        }
        if (lane < 2) piece[2 * wave + lane].rows = 0;
        while (at < end) {
            const SeqWork w = seq_work(a, b);
            const int64_t seq_places = w.places(a.Hk);
            if (at >= seq_at + seq_places) { seq_at += seq_places; ++b; continue; }
            const int unit = (int)((at - seq_at) / (w.tiles + 1));
            const int64_t unit_at = seq_at + (int64_t)unit * (w.tiles + 1);
            Run u;
            u.t0 = max((int)(at - unit_at) - 1, 0);
            u.t1 = (int)(end - unit_at - 1 < w.tiles ? end - unit_at - 1 : w.tiles);
            at = unit_at + w.tiles + 1;
            if (u.t0 >= u.t1) continue;                     // only the place before the tiles
            u.h = unit / w.row_tiles;
            u.row0 = (unit - u.h * w.row_tiles) * kRows;
            u.rows = min(kRows, w.q.n * a.group - u.row0);
            attend_run<DT, DP, WIDE>(a, b, w, u, x, token, head);
            if (u.t0 == 0 && u.t1 == w.tiles) store(w, u, x, token, head);
            else
                keep(w, u, x, 2 * wave + (u.t0 == 0 ? 1 : 0), unit_at,
                     1 + (int)((unit_at + w.tiles) / share / kWaves - (unit_at + 1) / share / kWaves));
        }
    } else {
        const int b = blockIdx.x, unit = blockIdx.y;
        const SeqWork w = seq_work(a, b);
        if (unit >= w.row_tiles * a.Hk) return;
        const int each = (w.tiles + kWaves - 1) / kWaves;
        Run u;
        u.t0 = wave * each;
        u.t1 = min(u.t0 + each, w.tiles);
        u.h = unit % a.Hk;
        u.row0 = unit / a.Hk * kRows;
        u.rows = min(kRows, w.q.n * a.group - u.row0);
        if (u.t0 >= u.t1) {
            if (lane == 0) piece[wave].rows = 0;
        } else {
            attend_run<DT, DP, WIDE>(a, b, w, u, x, token, head);
            if (w.tiles == 1) { store(w, u, x, token, head); return; }
            keep(w, u, x, wave, 0, 1);
        }
        if (w.tiles == 1) return;
    }

    // pieces of one unit lie next to each other, in order
    __syncthreads();
    bool told = false;
    for (int p0 = 0; p0 < kPieces;) {
        const Unit u = piece[p0];
        int p1 = p0 + 1;
        if (u.rows == 0) { p0 = p1; continue; }
        int ends = u.ends;
        for (int p = p1; p < kPieces; ++p) {
            if (piece[p].rows == 0) continue;
            if (piece[p].at != u.at) break;
            ends = piece[p].ends;
            p1 = p + 1;
        }
        const bool all = !SHARED || (u.begins && ends);
        float* out = SHARED ? part_of<DP>(a.work, gridDim.x, blockIdx.x, u.begins) : nullptr;
        if (SHARED && u.begins && !ends) {
            told = true;
            if (threadIdx.x == 0) reinterpret_cast<Unit*>(a.work)[blockIdx.x] = u;
        }
        const int quads = a.D / 4;
        for (int i = threadIdx.x; i < u.rows * quads; i += kThreads) {
            const int row = i / quads, d = i % quads * 4;
            Joined j{-__builtin_inff(), 0.0f, 0.0f};
            for (int p = p0; p < p1; ++p)
                if (piece[p].rows != 0) j.m = fmaxf(j.m, stat[p][row][0]);
            j.ref = j.m == -__builtin_inff() ? 0.0f : j.m;
            v4f o = {0.f, 0.f, 0.f, 0.f};
            for (int p = p0; p < p1; ++p)
                if (piece[p].rows != 0) {
                    const float f = __builtin_amdgcn_exp2f(stat[p][row][0] - j.ref);
                    j.l += stat[p][row][1] * f;
                    o += *reinterpret_cast<const v4f*>(&sums[p][row * RS + d]) * f;
                }
            if (all) {
                const int gr = u.row0 + row;
                store_row<DT>(a, u.token0 + gr / a.group, u.head * a.group + gr % a.group, d, o, j);
            } else {
                *reinterpret_cast<v4f*>(out + row * RS + 4 + d) = o;
                if (d == 0) { out[row * RS] = j.m; out[row * RS + 1] = j.l; }
            }
        }
        p0 = p1;
    }
    if (SHARED && threadIdx.x == 0 && !told) reinterpret_cast<Unit*>(a.work)[blockIdx.x].parts = 0;
}

template <int DT, int DP, bool WIDE>
hipError_t launch(const AttendArgs& a, hipStream_t stream)
{
    const int64_t rows = (int64_t)a.batch.max_q * a.group;
    if ((int64_t)a.batch.W * a.P <= kShortKeys) {
        const dim3 grid((unsigned)a.batch.B, (unsigned)((rows + kRows - 1) / kRows * a.Hk));
        hipLaunchKernelGGL((attend_rows_kernel<DT, DP, WIDE, false>), grid, dim3(waves_for(DP, false) * 64), 0,
                           stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((attend_rows_kernel<DT, DP, WIDE, true>), dim3(groups_for(DP)), dim3(kThreads), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    constexpr int groups = groups_for(DP);
    const Parts parts{reinterpret_cast<const Unit*>(a.work), part_of<DP>(a.work, groups, 0, true),
                      part_of<DP>(a.work, groups, 0, false), 2 * kRows * (DP + 4), 2 * kRows * (DP + 4)};
    // the parts that a unit has, about
    const int64_t units = a.batch.B * a.Hk * ((rows + kRows - 1) / kRows);
    return launch_join<DT, DP>(a, parts, groups, (int)(rows < kRows ? rows : kRows), (int)(groups / units), stream);
}

template <int DT, int DP>
hipError_t launch(const AttendArgs& a, hipStream_t stream)
{
    return a.P % kKeys == 0 ? launch<DT, DP, true>(a, stream) : launch<DT, DP, false>(a, stream);
}

template <int DT>
hipError_t launch(const AttendArgs& a, hipStream_t stream)
{
    if (a.D <= 64) return launch<DT, 64>(a, stream);
    if (a.D <= 128) return launch<DT, 128>(a, stream);
    if (a.D <= 192) return launch<DT, 192>(a, stream);
    return launch<DT, 256>(a, stream);
}

}  // namespace

hipError_t launch_paged_attention(const AttendArgs& a, int dtype, hipStream_t stream)
{
    if (attend_tiles(a)) return launch_attend_prompt(a, dtype, stream);
    return dtype == DT_BF16 ? launch<DT_BF16>(a, stream) : launch<DT_FP16>(a, stream);
}

int64_t attend_work_bytes(const AttendArgs& a)
{
    if (attend_tiles(a)) return attend_prompt_work_bytes(a);
    const int64_t dp = (a.D + 63) / 64 * 64;
    return groups_for((int)dp) * ((int64_t)sizeof(Unit) + 2 * kRows * (dp + 4) * 4);
}

}  // namespace fp8q
