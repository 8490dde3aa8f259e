// Attention over the paged FP8 cache for many query rows: a workgroup takes
// 128 rows (token, head of the group) of one key/value head, a wave 32 of them,
// and goes through the keys in tiles of 64 (see tile32.hpp for the arithmetic).
#include "tile32.hpp"

namespace fp8q {
namespace {

constexpr int kWaves = 4, kThreads = kWaves * 64, kWaveRows = 32, kTileRows = kWaves * kWaveRows;
constexpr int kLeastTiles = 4;            // of a part of a unit
constexpr int kRankedSeqs = 64;           // sequences that a wave ranks by length

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

    x.l += __shfl_xor(x.l, 32);
    if (!have_row) return;
    float* const part = parts_of<DP>(a, units) + ((place * a.Hk + h) * splits + split) * kPart<DP> +
                        (wave * kWaveRows + r) * (DP + 4);
    end_rows<DT, DP>(a, x, q.row + token, head, parts > 1 ? part : nullptr, hf);
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
