// Attention over the paged FP8 cache for many query rows: a workgroup takes
// 128 rows (token, head of the group) of one key/value head, a wave 32 of them,
// and goes through the keys in tiles of 64.
//
//   S^T = K Q^T   MFMA 32x32x16, keys along M, query rows along N
//   P   = 2^(S^T * ks + lv - m)   in the lane of its row
//   Y^T = V^T P   MFMA 32x32x16, channels along M
//
// The products run on 16-bit operands: E4M3 codes widen exactly to bf16 and
// fp16.  A lane of S^T holds 16 consecutive keys of one row for each 32 keys
// (the rows of K are put in LDS in the order that makes it so), which are the
// lane's part of the second product's operand, so P needs no exchange between
// lanes, and a row's maximum one.
#include "join.hpp"
#include "tile.hpp"

namespace fp8q {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kWaves = 4, kThreads = kWaves * 64, kWaveRows = 32, kTileRows = kWaves * kWaveRows;
constexpr int kKeys = 64;                 // keys of a tile
constexpr int kLeastTiles = 4;            // of a part of a unit
constexpr int kRankedSeqs = 64;           // sequences that a wave ranks by length

template <int DT>
__device__ __forceinline__ v16f mfma32(typename Half<DT>::vec a, v4i b, v16f c)
{
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, __builtin_bit_cast(v8b, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// 16 bytes for each active lane to lds_block + 16 * lane, asynchronously: from a buffer, or from any
// address.  Written as assembly because the compiler, which cannot tell the buffer being filled from
// the one being read, would wait for builtin loads of this kind before the next read of LDS, and no
// tile would be under way during the arithmetic.  They write no register; the kernel waits itself.
__device__ __forceinline__ uint32_t lds_address(const void* p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
__device__ __forceinline__ void buffer_to_lds(const v4i& rsrc, uint32_t lds_block, uint32_t offset)
{
    int m0;                               // kept for the compiler
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                 "buffer_load_dwordx4 %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "s"(uniform((int)lds_block)), "v"(offset), "s"(rsrc)
                 : "memory");
}
__device__ __forceinline__ void global_to_lds(const uint8_t* src, uint32_t lds_block)
{
    int m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "s"(uniform((int)lds_block)), "v"(src)
                 : "memory");
}
// The words of make_rsrc's resource.
__device__ __forceinline__ v4i rsrc_words(const uint8_t* base, int bytes)
{
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return v4i{uniform((int)(uint32_t)p), uniform((int)(uint32_t)(p >> 32)) & 0xffff, uniform(bytes), 0x00020000};
}

// Tiles in LDS.  Keys: row r of PITCH bytes is key 32 (r / 32) + key_of_row(r % 32), its 16-byte
// units exchanged by row.  Values: a channel's 64 bytes, units exchanged as by swz64.
__device__ __forceinline__ int key_of_row(int r) { return 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3); }
template <int DP>
struct Tile {
    static constexpr int kPitch = DP <= 64 ? 64 : (DP <= 128 ? 128 : 256);
    static constexpr int kUnits = kPitch / 16;
    static constexpr int kKeyBytes = kKeys * kPitch, kValueBytes = DP * kKeys;
    static constexpr int kKeyBlocks = kKeyBytes / 1024, kValueBlocks = kValueBytes / 1024;
    static __device__ __forceinline__ int swizzle(int row)
    {
        return kUnits == 4 ? (row >> 1) & 3 : row & (kUnits - 1);
    }
    static __device__ __forceinline__ int key_at(int row, int u) { return row * kPitch + ((u ^ swizzle(row)) << 4); }
};

__device__ __forceinline__ const uint8_t* shuffle(const uint8_t* p, int lane)
{
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)v, lane), hi = (uint32_t)__shfl((int)(v >> 32), lane);
    return reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ v4i value_at(const uint8_t* vt, int d, int tb, int r, int hf)
{
    return *reinterpret_cast<const v4i*>(vt + swz64(32 * d + r, 2 * tb + hf));
}
__device__ __forceinline__ void times16(v16f& sum, const v4i& v, const v8h (&w)[2])
{
    sum = mfma32<DT_FP16>(Half<DT_FP16>::widen(v[0], v[1]), __builtin_bit_cast(v4i, w[0]), sum);
    sum = mfma32<DT_FP16>(Half<DT_FP16>::widen(v[2], v[3]), __builtin_bit_cast(v4i, w[1]), sum);
}

// Values of keys that a row does not see must not count, but 0 * NaN would.  A tile that is not
// whole is looked through for codes of NaN; if there are any the wave goes on with a copy that has
// 0 for them, and notes the channels where a row does see one.
template <int DP>
__device__ __forceinline__ bool any_nan(const uint8_t* vt, int r, int hf)
{
    uint32_t any = 0;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            const v4i v = value_at(vt, d, tb, r, hf);
            any |= nan_bytes((uint32_t)v[0]) | nan_bytes((uint32_t)v[1]) | nan_bytes((uint32_t)v[2]) |
                   nan_bytes((uint32_t)v[3]);
        }
    return __ballot(any != 0) != 0;
}
template <int DP>
__device__ __forceinline__ void take_nan(uint32_t (&nan)[DP / 64], const uint8_t* vt, uint8_t* clean,
                                         const v8h (&seen)[2][2], int r, int hf)
{
    uint32_t got[DP / 64] = {};
#pragma unroll 1
    for (int d = DP / 32 - 1; d >= 0; --d) {               // 16 bits a time, the first channels last
        v16f hits;
#pragma unroll
        for (int i = 0; i < 16; ++i) hits[i] = 0.0f;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            v4i v = value_at(vt, d, tb, r, hf);
            times16(hits, nan_ones(v), seen[tb]);
            clear_nan(v);
            *reinterpret_cast<v4i*>(clean + swz64(32 * d + r, 2 * tb + hf)) = v;
        }
#pragma unroll
        for (int j = DP / 64 - 1; j > 0; --j) got[j] = got[j] << 16 | got[j - 1] >> 16;
        got[0] <<= 16;
#pragma unroll
        for (int i = 0; i < 16; ++i) got[0] |= hits[i] > 0.f ? 1u << i : 0u;
    }
#pragma unroll
    for (int j = 0; j < DP / 64; ++j) nan[j] |= got[j];
}

// The larger of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float max_halves(float v)
{
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

// What a wave has of its 32 query rows: lane (r, hf) half of row r's channels (32 d + 8 i + 4 hf ..),
// the row's reference, and its own keys' share of the denominator; a bit of `nan` for each channel
// that has seen NaN.
template <int DP>
struct Rows {
    v4i q[DP / 32][2];
    v16f acc[DP / 32];
    uint32_t nan[DP / 64];
    float m, l;
};

// A tile's terms.  whole: every row sees every key; clean: room for a tile of values.
template <int DT, int DP, bool WIDE>
__device__ __forceinline__ void add_tile(Rows<DP>& x, const uint8_t* kt, const PageScales& sc, const KeyRange& see,
                                         int key0, bool valid, bool whole, uint8_t* clean)
{
    using T = Tile<DP>;
    constexpr int NC = DP / 32, ND = DP / 32;
    const int lane = threadIdx.x & 63, r = lane & 31, hf = lane >> 5;
    const uint8_t* vt = kt + T::kKeyBytes;
    v16f s[2];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[tb][i] = 0.0f;
    // neighbouring matrix instructions add to different sums, so that none waits for the last
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        v4i k[2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) k[tb] = *reinterpret_cast<const v4i*>(kt + T::key_at(32 * tb + r, 2 * c + hf));
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int tb = 0; tb < 2; ++tb)
                s[tb] = mfma32<DT>(Half<DT>::widen(k[tb][2 * e], k[tb][2 * e + 1]), x.q[c][e], s[tb]);
    }
    if (!whole) {
        const bool on_page[2] = {WIDE ? valid : __shfl(valid ? 1 : 0, hf) != 0,
                                 WIDE ? valid : __shfl(valid ? 1 : 0, 2 + hf) != 0};
        v8h seen[2][2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            const int key = key0 + 32 * tb + 16 * hf, lo = see.lo - key, hi = on_page[tb] ? see.hi - key : 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool in = i >= lo && i < hi;
                s[tb][i] = in ? s[tb][i] : -__builtin_inff();
                seen[tb][i >> 3][i & 7] = in ? (_Float16)1.0f : (_Float16)0.0f;
            }
        }
        if (any_nan<DP>(vt, r, hf)) {
            take_nan<DP>(x.nan, vt, clean, seen, r, hf);
            vt = clean;
        }
    }
    // logarithms: a term is 2^(s * ks + lv), times the values' scale; one page a lane and block
    float ks[2], lv[2], top[2];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
        ks[tb] = WIDE ? sc.key : __shfl(sc.key, 2 * tb + hf);
        lv[tb] = WIDE ? sc.log_value : __shfl(sc.log_value, 2 * tb + hf);
        top[tb] = s[tb][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top[tb] = fmaxf(top[tb], s[tb][i]);
        top[tb] = __builtin_fmaf(top[tb], ks[tb], lv[tb]);
    }
    const float both = fmaxf(top[0], top[1]), highest = max_halves(both);
    if (__any(highest > x.m + kSlack)) {
        const float m1 = fmaxf(x.m, highest);
        const float alpha = m1 == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(x.m - m1);
        x.l *= alpha;
#pragma unroll
        for (int d = 0; d < ND; ++d) x.acc[d] *= alpha;
        x.m = m1;
    }
    const float ref = x.m == -__builtin_inff() ? 0.0f : x.m;
    v8h p[2][2];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
        const float offset = lv[tb] - (ref - kShift);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const v2f v = {__builtin_amdgcn_exp2f(__builtin_fmaf(s[tb][i], ks[tb], offset)),
                           __builtin_amdgcn_exp2f(__builtin_fmaf(s[tb][i + 1], ks[tb], offset))};
            sum += v[0];
            sum += v[1];
            const v2h w = __builtin_convertvector(v, v2h);
            p[tb][i >> 3][i & 7] = w[0];
            p[tb][i >> 3][(i & 7) + 1] = w[1];
        }
        x.l = __builtin_fmaf(sum, WIDE ? sc.inverse_value : __shfl(sc.inverse_value, 2 * tb + hf), x.l);
    }
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
        for (int d0 = 0; d0 < ND; d0 += 2) {
            const v4i v[2] = {value_at(vt, d0, tb, r, hf), value_at(vt, d0 + 1, tb, r, hf)};
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    x.acc[d0 + i] = mfma32<DT_FP16>(Half<DT_FP16>::widen(v[i][2 * e], v[i][2 * e + 1]),
                                                    __builtin_bit_cast(v4i, p[tb][e]), x.acc[d0 + i]);
        }
}

// The workgroups of a key/value head take units of kTileRows rows of one sequence; this gives the
// `place`-th one its sequence and first row.  Places follow each other as the workgroups start: the
// first kFirst go to a compute unit each, the next kFirst join them, the others follow where one
// ends.  Under a causal mask a unit's time is its last position, so the longest units come first,
// then the shortest, so that every compute unit has one of both, then the rest.
__device__ __forceinline__ int64_t rank_of(int64_t place, int64_t count, int first)
{
    if (place < first) return place;
    if (place < 2 * (int64_t)first) return count - 1 - (place - first);
    return place - first;
}
__device__ __forceinline__ bool find_unit(const AttendArgs& a, int64_t place, int splits, int64_t units, int* lds,
                                          int& b, int& row0)
{
    const PagedBatch& s = a.batch;
    const int first = (kCUs + a.Hk * splits - 1) / (a.Hk * splits), lane = threadIdx.x & 63;
    if (s.B <= kRankedSeqs) {
        // ranked by the sequences' lengths, the last rows of each first
        PagedSeq q{0, 0, 0, 0};
        if (lane < s.B) q = paged_seq(s, lane, a.P);
        const int tiles = (int)(((int64_t)q.n * a.group + kTileRows - 1) / kTileRows);
        int before = 0, count = 0;
        for (int k = 0; k < s.B; ++k) {
            const int t = __builtin_amdgcn_readlane(tiles, k), len = __builtin_amdgcn_readlane(q.len, k);
            before += len > q.len || (len == q.len && k < lane) ? t : 0;
            count += t;
        }
        if (place >= count) return false;
        const int rank = (int)rank_of(place, count, first);
        const uint64_t here = __ballot(rank >= before && rank < before + tiles);
        b = (int)__builtin_ctzll(here);
        row0 = (__builtin_amdgcn_readlane(tiles, b) - 1 - (rank - __builtin_amdgcn_readlane(before, b))) * kTileRows;
        return true;
    }
    // in the sequences' order; those of sequence b begin at unit q_start[b] * group / kTileRows + b
    if (place >= units) return false;
    const int64_t u = units - 1 - rank_of(place, units, first);
    int below = 0;
    for (int k = threadIdx.x; k < s.B; k += kThreads)
        below += (int64_t)clamp_int(s.q_start[k], 0, s.T) * a.group / kTileRows + k <= u ? 1 : 0;
    b = uniform(max(block_sum_int<kThreads>(below, lds) - 1, 0));
    const PagedSeq q = paged_seq(s, b, a.P);
    const int64_t row = (u - ((int64_t)q.row * a.group / kTileRows + b)) * kTileRows;
    row0 = (int)row;
    return row >= 0 && row < (int64_t)q.n * a.group;
}

// The scratch where units are cut: what each is, then its parts.
template <int DP>
constexpr int64_t kPart = kTileRows * (DP + 4);
template <int DP>
__host__ __device__ __forceinline__ float* parts_of(const AttendArgs& a, int64_t units)
{
    return a.work + units * a.Hk * (int64_t)(sizeof(Unit) / 4);
}

template <int DT, int DP, bool WIDE>
__global__ void __launch_bounds__(kThreads, DP <= 128 ? 2 : 1)
    attend_prompt_kernel(const AttendArgs a, int64_t units, int splits)
{
    using T = Tile<DP>;
    constexpr int NC = DP / 32, ND = DP / 32;
    constexpr int KB = T::kKeyBlocks / kWaves, VB = T::kValueBlocks / kWaves;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][T::kKeyBytes + T::kValueBytes];
    __shared__ __attribute__((aligned(16))) uint8_t clean[kWaves][T::kValueBytes];
    __shared__ int found[kWaves];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), r = lane & 31, hf = lane >> 5;
    const int64_t index = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int h = (int)(index % a.Hk);
    int b, row0;
    const int64_t place = index / a.Hk / splits;
    const int split = (int)(index / a.Hk % splits);
    Unit* const told = reinterpret_cast<Unit*>(a.work) + place * a.Hk + h;
    if (place >= units) return;
    if (!find_unit(a, place, splits, units, found, b, row0)) {
        if (splits > 1 && split == 0 && tid == 0) told->parts = 0;
        return;
    }
    const PagedSeq q = paged_seq(a.batch, b, a.P);
    const int rows = min(q.n * a.group - row0, kTileRows);

    const int wave_row0 = row0 + wave * kWaveRows;
    const int my_row = wave_row0 + r, token = my_row / a.group, head = h * a.group + my_row % a.group;
    const bool have_row = my_row < row0 + rows;
    KeyRange see = key_range(a, q, token);
    if (!have_row) see.lo = see.hi = 0;
    const KeyRange first = key_range(a, q, row0 / a.group), last = key_range(a, q, (row0 + rows - 1) / a.group);
    const bool idle = wave_row0 >= row0 + rows;
    const int wave_last = min(wave_row0 + kWaveRows, row0 + rows) - 1;
    const KeyRange wfirst = key_range(a, q, wave_row0 / a.group), wlast = key_range(a, q, wave_last / a.group);
    int t0 = first.lo / kKeys, t1 = (last.hi + kKeys - 1) / kKeys, parts = 1;
    if (splits > 1) {
        const int each = max((t1 - t0 + splits - 1) / splits, kLeastTiles);
        parts = max((t1 - t0 + each - 1) / each, 1);
        if (split == 0 && tid == 0)
            *told = Unit{0, parts > 1 ? parts : 0, 1, 1, q.row, h, row0, rows, 0};
        if (split >= parts) return;
        t0 += split * each;
        t1 = min(t0 + each, t1);
    }

    Rows<DP> x;
    {
        const uint16_t* src = a.q + (int64_t)(q.row + token) * a.q_stride + (int64_t)head * a.D;
        const v4i zero = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = 32 * c + 16 * hf;
            const bool have = have_row && d < a.D;
            x.q[c][0] = have ? *reinterpret_cast<const v4i*>(src + d) ^ a.q_flip : zero;
            x.q[c][1] = have ? *reinterpret_cast<const v4i*>(src + d + 8) ^ a.q_flip : zero;
        }
    }
    if (!WIDE && a.D < T::kPitch) {       // channels that no load fills
        for (int i = tid; i < 2 * T::kKeyBytes / 16; i += kThreads)
            *reinterpret_cast<v4i*>(&lds[i / (T::kKeyBytes / 16)][i % (T::kKeyBytes / 16) * 16]) = v4i{0, 0, 0, 0};
        __syncthreads();
    }

    // A tile's keys in four groups of 16, each on one page; lane i of a wave keeps what is known of
    // group i % 4 (where a page holds whole tiles all lanes the same).
    const uint32_t page_bytes = (uint32_t)(a.P * a.D), pool_stride = (uint32_t)a.Hk * page_bytes;
    const int group_key = WIDE ? 0 : 16 * (lane & 3);
    const uint8_t* const kbase = a.k_pages + (uint32_t)h * page_bytes;
    const uint8_t* const vbase = a.v_pages + (uint32_t)h * page_bytes;
    const uint32_t lds_at = lds_address(&lds[0][0]);
    const auto load_tile = [&](const PageRef& p, uint32_t dst) {
        if constexpr (WIDE) {
            // the tile is on one page: a lane's offsets are the same in every tile; channels past D
            // are out of the buffer's range (values) or sent there (keys) and become 0
            const uint64_t at = (uint64_t)(uint32_t)uniform((int)p.page) * pool_stride;
            const uint32_t inside = (uint32_t)uniform(p.inside);
            const v4i rk = rsrc_words(kbase + at + inside * (uint32_t)a.D, kKeys * a.D);
            const v4i rv = rsrc_words(vbase + at + inside, (int)(page_bytes - inside));
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const int unit = (wave * KB + j) * 64 + lane, row = unit / T::kUnits;
                const int c = (unit % T::kUnits) ^ T::swizzle(row), key = (row & 32) + key_of_row(row & 31);
                buffer_to_lds(rk, dst + (wave * KB + j) * 1024, 16 * c < a.D ? (uint32_t)(key * a.D + 16 * c) : kOOB);
            }
#pragma unroll
            for (int j = 0; j < VB; ++j) {
                const int d = (wave * VB + j) * 16 + (lane >> 2), g = (lane & 3) ^ ((d >> 1) & 3);
                buffer_to_lds(rv, dst + T::kKeyBytes + (wave * VB + j) * 1024, (uint32_t)(d * a.P + 16 * g));
            }
        } else {
            const uint64_t at = (uint64_t)(uint32_t)p.page * pool_stride;
            const uint8_t* const kp = kbase + at + (uint32_t)(p.inside * a.D);
            const uint8_t* const vp = vbase + at + (uint32_t)p.inside;
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const int unit = (wave * KB + j) * 64 + lane, row = unit / T::kUnits;
                const int c = (unit % T::kUnits) ^ T::swizzle(row), key = (row & 32) + key_of_row(row & 31);
                const uint8_t* src = shuffle(kp, key >> 4) + (key & 15) * a.D + 16 * c;
                if (16 * c < a.D) global_to_lds(src, dst + (wave * KB + j) * 1024);
            }
#pragma unroll
            for (int j = 0; j < VB; ++j) {
                const int d = (wave * VB + j) * 16 + (lane >> 2), g = (lane & 3) ^ ((d >> 1) & 3);
                const uint8_t* src = shuffle(vp, g) + d * a.P;
                if (d < a.D) global_to_lds(src, dst + T::kKeyBytes + (wave * VB + j) * 1024);
            }
        }
    };

#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) x.acc[d][i] = 0.0f;
#pragma unroll
    for (int d = 0; d < DP / 64; ++d) x.nan[d] = 0u;
    x.m = -__builtin_inff();
    x.l = 0.0f;

    // A tile's codes are requested a tile ahead.  WIDE: lane i of a wave keeps what is known of the
    // tile's page with the i-th of 64 tiles, loaded when the first of them is requested.
    PageRef many{0, 0, false};
    PageScales many_scales{};
    uint64_t many_valid = 0;
    const auto look_up = [&](int t) {
        const int key = (t + lane) * kKeys;
        many = page_ref(a, b, q.len, key);
        many_scales = page_scales(a, many.page, h);
        many_valid = __ballot(many.valid);
    };
    // Else its scales as well, and its pages' ids two tiles ahead.  What is loaded to registers is
    // requested before the codes and not touched before the next tile: loads return in order, and a
    // use would wait for the codes as well.
    const auto id_of = [&](int t) { return page_id(a, b, q.len, t * kKeys + group_key); };
    int next_id = 0;
    bool next_valid = false;
    float next_k = 0.0f, next_v = 0.0f;
    const auto request = [&](int t, uint32_t dst) {
        if constexpr (WIDE) {
            const int i = (t - t0) & 63;
            if (i == 0) look_up(t);
            load_tile(PageRef{__builtin_amdgcn_readlane((int)many.page, i), (t * kKeys) & (a.P - 1), true}, dst);
        } else {
            const PageRef next = page_ref(a, next_id, t * kKeys + group_key);
            const int64_t cell = next.page * a.Hk + h;
            next_valid = next.valid;
            next_k = a.k_scale[cell];
            next_v = a.v_scale[cell];
            next_id = id_of(t + 1);
            load_tile(next, dst);
        }
    };
    if (!WIDE) next_id = id_of(t0);
    if (t0 < t1) request(t0, lds_at);
    for (int t = t0; t < t1; ++t) {
        const int at = (t - t0) & 1;
        const uint8_t* const kt = lds[at];
        wait_vm<0>();
        if (!WIDE) asm volatile("" : "+v"(next_k), "+v"(next_v), "+v"(next_id));
        __syncthreads();                  // tile t is there, and tile t - 1 has been read
        PageScales now;
        bool valid;
        if constexpr (WIDE) {
            const int i = (t - t0) & 63;
            const auto lane_i = [&](float v) {
                return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i));
            };
            now = PageScales{lane_i(many_scales.key), lane_i(many_scales.log_value), lane_i(many_scales.inverse_value)};
            valid = (many_valid >> i & 1) != 0;
        } else {
            now = page_scales(a, next_k, next_v);
            valid = next_valid;
        }
        if (t + 1 < t1) request(t + 1, lds_at + (at ^ 1) * (uint32_t)sizeof(lds[0]));
        const int key0 = t * kKeys;
        if (idle || key0 >= wlast.hi || key0 + kKeys <= wfirst.lo) continue;   // no row of this wave sees the tile

        const bool whole = wfirst.lo <= key0 && wlast.lo <= key0 && wfirst.hi >= key0 + kKeys &&
                           wlast.hi >= key0 + kKeys && __all(valid);
        add_tile<DT, DP, WIDE>(x, kt, now, see, key0, valid, whole, clean[wave]);
    }

    x.l += __shfl_xor(x.l, 32);
    if (!have_row) return;
    const Joined j{x.m, x.m == -__builtin_inff() ? 0.0f : x.m, x.l};
    float* const part = parts_of<DP>(a, units) + ((place * a.Hk + h) * splits + split) * kPart<DP> +
                        (wave * kWaveRows + r) * (DP + 4);
    if (parts > 1 && hf == 0) { part[0] = x.m; part[1] = x.l; }
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = 32 * d + 8 * e + 4 * hf;
            v4f o;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = (x.nan[d >> 1] >> (16 * (d & 1) + 4 * e + i) & 1u) != 0 ? __builtin_nanf("") : x.acc[d][4 * e + i];
            if (c >= a.D) continue;
            if (parts > 1) *reinterpret_cast<v4f*>(part + 4 + c) = o;
            else store_row<DT>(a, q.row + token, head, c, o, j);
        }
}

// Units of all sequences at most, and into how many parts of the keys each is cut: as many as make
// one round of the workgroups that the chip holds at once.
struct Cut {
    int64_t units;
    int splits;
};
Cut cut_of(const AttendArgs& a)
{
    const int64_t loose = (int64_t)a.batch.T * a.group / kTileRows + a.batch.B;
    const int64_t tight = a.batch.B * (((int64_t)a.batch.max_q * a.group + kTileRows - 1) / kTileRows);
    const int64_t units = loose < tight ? loose : tight, slots = kCUs * (a.D <= 128 ? 2 : 1);
    const int64_t tiles = ((int64_t)a.batch.W * a.P + kKeys - 1) / kKeys, most = (tiles + kLeastTiles - 1) / kLeastTiles;
    int64_t splits = slots / (units * a.Hk);
    splits = splits < most ? splits : most;
    return Cut{a.batch.B <= kRankedSeqs ? units : loose, (int)(splits < 1 ? 1 : splits > kMostParts ? kMostParts : splits)};
}

template <int DT, int DP, bool WIDE>
hipError_t launch(const AttendArgs& a, hipStream_t stream)
{
    const Cut cut = cut_of(a);
    const int64_t groups = cut.units * a.Hk * cut.splits, most = max_groups(kThreads), gx = groups < most ? groups : most;
    hipLaunchKernelGGL((attend_prompt_kernel<DT, DP, WIDE>), dim3((unsigned)gx, (unsigned)((groups + gx - 1) / gx)),
                       dim3(kThreads), 0, stream, a, cut.units, cut.splits);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || cut.splits == 1) return e;
    const float* const parts = parts_of<DP>(a, cut.units);
    return launch_join<DT, DP>(a, Parts{reinterpret_cast<const Unit*>(a.work), parts, parts, cut.splits * kPart<DP>, kPart<DP>},
                               (int)(cut.units * a.Hk), kTileRows, cut.splits, stream);
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

int64_t attend_prompt_work_bytes(const AttendArgs& a)
{
    const Cut cut = cut_of(a);
    if (cut.splits == 1) return 16;
    const int64_t dp = (a.D + 63) / 64 * 64;
    return cut.units * a.Hk * ((int64_t)sizeof(Unit) + cut.splits * kTileRows * (dp + 4) * 4);
}

hipError_t launch_attend_prompt(const AttendArgs& a, int dtype, hipStream_t stream)
{
    return dtype == DT_BF16 ? launch<DT_BF16>(a, stream) : launch<DT_FP16>(a, stream);
}

}  // namespace fp8q
