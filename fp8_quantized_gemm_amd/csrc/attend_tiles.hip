// Attention over the paged FP8 cache for many query rows or long sequences: a
// workgroup takes 128 rows (token, head of the group) of one key/value head, a
// wave 32 of them, and goes through the keys in tiles of 64 (see tile32.hpp for
// the arithmetic).  A tile's codes go to LDS once for the four waves, the next
// tile's on the way during the arithmetic; two workgroups share a compute unit.
//
// Prompts are bound by the vector units: a tile takes a wave 32 MFMAs and about
// 330 other instructions, of which 128 widen codes and 150 are the softmax.  4096
// tokens with 64/8 heads x 128 take 293 us, 0.94 PFLOP/s (a library product of
// 8192^3 reaches 1.2), vector units busy 70% and matrix units 43% of the time;
// 2048 with 32/32 heads 55 us, where one workgroup of a compute unit's two ends
// early.  Decoding few long sequences is bound by HBM: 1 of 131072 (268 MB) in
// 512 parts 54 us and 6 to join them.  (Calls on a busy stream; after a pause
// they take up to a sixth longer, until the clocks have risen.)
#include "tile32.hpp"

namespace fp8q {
namespace {

constexpr int kWaves = 4, kThreads = kWaves * 64, kWaveRows = 32, kTileRows = kWaves * kWaveRows;
// Workgroups that the chip holds at once.
constexpr int slots_for(int dp) { return kCUs * (dp <= 128 ? 2 : 1); }
constexpr int kRankedSeqs = 64;           // sequences that a wave ranks by length

// Rows of a part of a unit.
__host__ __device__ __forceinline__ int part_rows(const AttendArgs& a)
{
    const int64_t rows = (int64_t)a.batch.max_q * a.group;
    return (int)(rows < kTileRows ? rows : kTileRows);
}
// Key tiles that a part has at least: its rows go through the scratch.  Where units are few, parts of
// 4 tiles are short enough to use the chip (64/8 heads, 128 tokens of 2000: 31 us, 36 with 20), and for
// few rows parts of 2 (here 1 token of 2000 14.0 us, 16.4 with 4; but 256 of 256: 21.1 us, 14.3 with 4).
// Where they are more than a quarter of the workgroups that fit, cutting them doubles those on a
// compute unit at best, which pays for many rows if the parts are long (512 of 512: 22 us, 33 with 4).
__host__ __device__ __forceinline__ int least_tiles(const AttendArgs& a, int64_t units, int slots)
{
    const int rows = part_rows(a);
    if (units * a.Hk * 4 > slots) return 4 + rows / 8;
    return rows <= kWholeRows ? 2 : 4;
}

// What a workgroup does: rows row0 .. of sequence b, the `part`-th of `parts` equal runs of the keys
// that they see.
struct Item {
    int b, row0, part, parts;
    int64_t unit, units;                  // of the key/value head: this one, and how many there are
};

// The workgroups of a key/value head take the units of all sequences (kTileRows rows each), in parts
// where the units are fewer than the workgroups that fit the chip; this is the `place`-th one's item.
//
// Up to kRankedSeqs sequences every wave looks at all of them, one a lane.  They are ranked by their
// lengths, the last rows of each first: under a causal mask a unit's time is its last position.
// `cut`: a sequence's units get so many parts that each part has about the same number of key tiles,
// the least for which the parts still fit.  Not cut: units follow each other as workgroups start, the
// first `first` to a compute unit each, the next join them, the others follow where one ends; so the
// longest come first, then the shortest, so that every compute unit has one of both, then the rest.
//
// More sequences are taken in their order, and every unit has `splits` parts.  Units are numbered in
// the way that needs fewer numbers: as many for each sequence as max_q allows, or those of sequence b
// from q_start[b] * group / kTileRows + b on.
__host__ __device__ __forceinline__ int64_t loose_units(const AttendArgs& a)
{
    return (int64_t)a.batch.T * a.group / kTileRows + a.batch.B;
}
__host__ __device__ __forceinline__ int most_units(const AttendArgs& a)           // of a sequence
{
    return (int)(((int64_t)a.batch.max_q * a.group + kTileRows - 1) / kTileRows);
}
__device__ __forceinline__ int64_t rank_of(int64_t place, int64_t count, int first)
{
    if (place < first) return place;
    if (place < 2 * (int64_t)first) return count - 1 - (place - first);
    return place - first;
}
__device__ __forceinline__ float wave_total(float v)
{
#define FP8Q_DPP_ADD(ctrl, rows) \
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, rows, 0xf, false))
    FP8Q_DPP_ADD(0xB1, 0xf);   // quad_perm [1,0,3,2]
    FP8Q_DPP_ADD(0x4E, 0xf);   // quad_perm [2,3,0,1]
    FP8Q_DPP_ADD(0x141, 0xf);  // row_half_mirror
    FP8Q_DPP_ADD(0x140, 0xf);  // row_mirror
    FP8Q_DPP_ADD(0x142, 0xa);  // row_bcast15 -> rows 1, 3
    FP8Q_DPP_ADD(0x143, 0xc);  // row_bcast31 -> rows 2, 3: lane 63 holds the sum
#undef FP8Q_DPP_ADD
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ bool find_item(const AttendArgs& a, int64_t place, bool cut, int splits, int slots,
                                          int64_t units, int* lds, Item& item)
{
    const PagedBatch& s = a.batch;
    const int first = (kCUs + a.Hk - 1) / a.Hk, lane = threadIdx.x & 63;
    if (s.B <= kRankedSeqs) {
        PagedSeq q{0, 0, 0, 0};
        if (lane < s.B) q = paged_seq(s, lane, a.P);
        const int tiles = (int)(((int64_t)q.n * a.group + kTileRows - 1) / kTileRows);
        int parts = 1;
        if (cut) {
            // a unit's key tiles, as those of the sequence's middle token
            const KeyRange mid = key_range(a, q, q.n / 2);
            const int keys = (mid.hi - mid.lo) / kKeys + 1, most = slots / a.Hk;
            int each = max((int)ceilf(wave_total((float)tiles * (float)keys) / (float)most), least_tiles(a, units, slots));
            // twice the even share is always enough, as the units are half of what fits at most
            for (int i = 0; i < 13; ++i) {
                parts = (keys + each - 1) / each;
                if (wave_total((float)tiles * (float)parts) <= (float)most) break;
                each += (each + 15) >> 4;
                parts = 1;
            }
        }
        int before = 0, count = 0, units_before = 0;
        item.units = 0;
        for (int k = 0; k < s.B; ++k) {
            const int t = __builtin_amdgcn_readlane(tiles, k), p = t * __builtin_amdgcn_readlane(parts, k);
            const int len = __builtin_amdgcn_readlane(q.len, k);
            const bool ahead = len > q.len || (len == q.len && k < lane);
            before += ahead ? p : 0;
            units_before += ahead ? t : 0;
            count += p;
            item.units += t;
        }
        if (place >= count) return false;
        const int rank = cut ? (int)place : (int)rank_of(place, count, first);
        const int b = (int)__builtin_ctzll(__ballot(rank >= before && rank < before + tiles * parts));
        const int i = rank - __builtin_amdgcn_readlane(before, b);
        item.b = b;
        item.parts = __builtin_amdgcn_readlane(parts, b);
        item.part = i % item.parts;
        const int u = i / item.parts;
        item.unit = __builtin_amdgcn_readlane(units_before, b) + u;
        item.row0 = (__builtin_amdgcn_readlane(tiles, b) - 1 - u) * kTileRows;
        return true;
    }
    item.units = 0;                       // every unit that is not there is told by its first part
    item.unit = place / splits;
    const int64_t u = units - 1 - (cut ? item.unit : rank_of(place, units, first));
    item.parts = splits;
    item.part = (int)(place % splits);
    int64_t first_unit;
    if (most_units(a) * (int64_t)s.B <= loose_units(a)) {
        item.b = (int)(u / most_units(a));
        first_unit = (int64_t)item.b * most_units(a);
    } else {
        int below = 0;
        for (int k = threadIdx.x; k < s.B; k += kThreads)
            below += (int64_t)clamp_int(s.q_start[k], 0, s.T) * a.group / kTileRows + k <= u ? 1 : 0;
        item.b = uniform(max(block_sum_int<kThreads>(below, lds) - 1, 0));
        first_unit = (int64_t)clamp_int(s.q_start[item.b], 0, s.T) * a.group / kTileRows + item.b;
    }
    const PagedSeq q = paged_seq(s, item.b, a.P);
    const int64_t row = (u - first_unit) * kTileRows;
    item.row0 = (int)row;
    return row >= 0 && row < (int64_t)q.n * a.group;
}

// The scratch where units are cut: what each unit of each key/value head is, then a part for each
// workgroup.
__host__ __device__ __forceinline__ float* parts_of(const AttendArgs& a, int64_t units)
{
    static_assert(sizeof(Unit) % 16 == 0, "parts are read 16 bytes at a time");
    return a.work + units * a.Hk * (int64_t)(sizeof(Unit) / 4);
}

template <int DT, int DP, bool WIDE>
__global__ void __launch_bounds__(kThreads, DP <= 128 ? 2 : 1)
    attend_tiles_kernel(const AttendArgs a, int64_t units, int64_t groups, int splits, int cut)
{
    using T = Tile<DP>;
    constexpr int KB = T::kKeyBlocks / kWaves, VB = T::kValueBlocks / kWaves;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][T::kKeyBytes + T::kValueBytes];
    __shared__ __attribute__((aligned(16))) uint8_t clean[kWaves][T::kValueBytes];
    __shared__ int found[kWaves];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), r = lane & 31, hf = lane >> 5;
    const int64_t index = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int h = (int)(index % a.Hk);
    Item item;
    if (index >= groups) return;
    const int64_t place = index / a.Hk;
    const bool have = find_item(a, place, cut != 0, splits, slots_for(DP), units, found, item);
    Unit* const told = reinterpret_cast<Unit*>(a.work);
    if (cut && tid == 0) {
        // units that the batch might have had, but has not
        if (a.batch.B <= kRankedSeqs ? place >= item.units && place < units : !have && item.part == 0)
            told[(a.batch.B <= kRankedSeqs ? place : item.unit) * a.Hk + h].parts = 0;
    }
    if (!have) return;
    const int b = item.b, row0 = item.row0;
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
    int t0 = first.lo / kKeys, t1 = (last.hi + kKeys - 1) / kKeys;
    if (cut) {
        // a part that gets no tile has sums of nothing, which join like others
        const int each = (t1 - t0 + item.parts - 1) / item.parts;
        if (tid == 0 && item.part == 0 && item.unit < units)
            told[item.unit * a.Hk + h] =
                Unit{(int)index, item.parts > 1 ? item.parts : 0, q.row, h, row0, rows, {0, 0}};
        t0 = min(t0 + item.part * each, t1);
        t1 = min(t0 + each, t1);
    }

    Rows<DP> x;
    begin_rows<DP>(a, x, have_row, q.row + token, head, hf);
    if (!WIDE && a.D < T::kPitch) {
        clear_lds(&lds[0][0], (int)sizeof(lds), tid, kThreads);
        __syncthreads();
    }

    // a tile's codes are requested a tile ahead
    const uint32_t lds_at = lds_address(&lds[0][0]);
    Pages pages{};
    const auto request = [&](int t, int slot) {
        const int i = (t - t0) % kLookUp<WIDE>;
        if (i == 0) pages = look_up<WIDE>(a, b, q.len, t * kKeys, h);
        request_tile<DP, WIDE, KB, VB>(a, pages, i, t * kKeys, h, wave, lds_at + slot * (uint32_t)sizeof(lds[0]));
        if (i == 0) x.apart |= any_apart(pages.sc);
    };
    if (t0 < t1) request(t0, 0);
    for (int t = t0; t < t1; ++t) {
        const int slot = (t - t0) & 1;
        wait_vm<0>();
        __syncthreads();                  // tile t is there, and tile t - 1 has been read
        bool valid;
        const PageScales now = tile_scales<WIDE>(pages, (t - t0) % kLookUp<WIDE>, valid);
        if (t + 1 < t1) request(t + 1, slot ^ 1);
        const int key0 = t * kKeys;
        if (idle || key0 >= wlast.hi || key0 + kKeys <= wfirst.lo) continue;   // no row of this wave sees the tile

        const bool whole = wfirst.lo <= key0 && wlast.lo <= key0 && wfirst.hi >= key0 + kKeys &&
                           wlast.hi >= key0 + kKeys && __all(valid);
        add_tile<DT, DP, WIDE>(x, lds[slot], now, see, key0, valid, whole, clean[wave]);
    }

    join_lanes(x.z, x.l, 32);
    if (!have_row) return;
    float* const part = parts_of(a, units) + (index * part_rows(a) + wave * kWaveRows + r) * (DP + 4);
    end_rows<DT, DP>(a, x, q.row + token, head, item.parts > 1 ? part : nullptr, hf);
}

// Units of all sequences at most; workgroups; whether units are cut, and into how many parts each
// where the kernel does not choose.
struct Plan {
    int64_t units, groups;
    int splits;
    bool cut;
};
Plan plan_of(const AttendArgs& a)
{
    const int64_t loose = loose_units(a), even = (int64_t)a.batch.B * most_units(a);
    const int64_t units = loose < even ? loose : even, slots = slots_for((int)a.D);
    const int64_t tiles = ((int64_t)a.batch.W * a.P + kKeys - 1) / kKeys, least = least_tiles(a, units, (int)slots);
    const bool cut = units * a.Hk * 2 <= slots && tiles > least;
    if (a.batch.B <= kRankedSeqs)
        return cut ? Plan{units, slots / a.Hk * a.Hk, 1, true} : Plan{units, units * a.Hk, 1, false};
    const int64_t fit = cut ? slots / (units * a.Hk) : 1, most = (tiles + least - 1) / least;
    const int64_t splits = fit < most ? fit : most;
    return Plan{units, units * a.Hk * splits, (int)splits, cut};
}

template <int DT, int DP, bool WIDE>
hipError_t launch(const AttendArgs& a, hipStream_t stream)
{
    const Plan plan = plan_of(a);
    const int64_t groups = plan.groups, most = max_groups(kThreads), gx = groups < most ? groups : most;
    hipLaunchKernelGGL((attend_tiles_kernel<DT, DP, WIDE>), dim3((unsigned)gx, (unsigned)((groups + gx - 1) / gx)),
                       dim3(kThreads), 0, stream, a, plan.units, groups, plan.splits, plan.cut ? 1 : 0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !plan.cut) return e;
    return launch_join<DT, DP>(a, parts_of(a, plan.units), plan.units, part_rows(a), stream);
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

int64_t attend_tiles_work_bytes(const AttendArgs& a)
{
    const Plan plan = plan_of(a);
    if (!plan.cut) return 16;
    const int64_t dp = (a.D + 63) / 64 * 64;
    return plan.units * a.Hk * (int64_t)sizeof(Unit) + plan.groups * part_rows(a) * (dp + 4) * 4;
}

hipError_t launch_attend_tiles(const AttendArgs& a, int dtype, hipStream_t stream)
{
    return dtype == DT_BF16 ? launch<DT_BF16>(a, stream) : launch<DT_FP16>(a, stream);
}

}  // namespace fp8q
