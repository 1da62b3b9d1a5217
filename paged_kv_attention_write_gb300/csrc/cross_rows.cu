// cross_rows.cu -- few query rows over another sequence's whole paged context, each within its own
// range of keys (kernels: stream_rows.cuh), and the choice between them and the chunks' kernel.
#include "cross.cuh"
#include "stream_rows.cuh"

namespace pa {
namespace {

int launch_cross_rows(const CrossArgs &c) {
    const PrefillArgs &a = c.a;
    Params p{};
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.query = a.query;
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.max_blocks_per_seq = a.max_blocks_per_seq;
    p.max_context_len = a.max_context_len;
    p.num_heads = a.num_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.group = a.num_heads / a.num_kv_heads;
    p.block_size = a.block_size;
    p.num_blocks = a.num_blocks;
    p.qk_scale_log2 = a.scale * kLog2e;
    p.status = a.status;
    p.query_start_loc = a.query_start_loc;
    p.key_ranges = c.key_ranges;
    p.num_tokens = a.num_tokens;
    p.max_query_len = a.max_query_len;
    p.num_seqs = a.num_seqs;
    p.group_log2 = p.group == 1 ? 0 : p.group == 2 ? 1 : p.group == 4 ? 2 : 3;
    p.tokens = 1;
    const int longest = std::min(a.max_query_len, a.num_tokens);
    // fp32: a warp holds four columns, so eight take two warps per key and nothing is gained by sharing
    // the keys (19 sequences of 1 to 3 rows of 4 heads 23.4 us with two rows to an item, 17.5 with one)
    const int fill = a.kv_dtype == PA_F32 ? 4 : 8;
    while (p.tokens < longest && p.tokens * p.group < fill) p.tokens *= 2;
    p.token_groups = (longest - 1) / p.tokens + 1;
    const int columns = p.tokens * p.group;
    // Clusters as in decode_window.cu: the CTAs of one full wave, none with less than one stage of
    // keys (two past eight CTAs).
    const int sms = std::max(1, device_sm_count());
    const int64_t slots = 2 * sms, most = a.max_context_len;
    const int64_t stage_keys = 16384 / (a.head_dim * (a.kv_dtype == PA_F32 ? 4 : 2));
    const int64_t items = (int64_t)a.num_seqs * p.token_groups * a.num_kv_heads;
    // those that have rows: of ragged sequences some items are empty and gone at once
    const int64_t live = std::min<int64_t>(items, (p.tokens == 1 ? a.num_tokens : a.num_tokens / p.tokens + (int64_t)a.num_seqs) *
                                                      a.num_kv_heads);
    auto fit = [&](int size) { return slots * (size <= 2 ? 64 : size == 4 ? 63 : size == 8 ? 61 : 48) / 64; };
    int cluster = 1;
    while (cluster < 16 && live * cluster * 2 <= fit(cluster * 2) &&
           most > stage_keys * cluster * (cluster < 8 ? 1 : 2))
        cluster *= 2;
    // Past a wave, in twos where some items have no rows (sequences of 1 to 3 and 1 to 8 fp32 rows): their CTAs
    // are gone at once and leave the others unevenly on the SMs, whole items more than halves.  Against whole
    // items, 156 to 208 with rows among 216 to 320 in all: contexts of 0 to 1500 keys 0.60 to 0.80 of the
    // time, 0 to 4000 0.55 to 0.62, 3000 to 4000 0.82 to 0.98, all of 4000 0.94 to 1.06, all of 1500 1.02 to
    // 1.24; all of 1000 1.10 to 1.31, which is too much; 240 to 256 items of 0 to 1500 keys 0.76 to 0.99, all of
    // 1500 1.10 to 1.23.  Without such items twos lose where contexts are alike (176 items of 1500 keys
    // 28 -> 39 us, of 4000 64 -> 82; of 0 to 4000 60 -> 41).
    if (cluster == 1 && live < items && live * 3 <= slots * 2 && most > 1024) cluster = 2;
    p.unit = cluster > 1 || most >= 64 * (int64_t)a.block_size ? a.block_size / 8 : 1;
    const int per_sm = (int)std::min<int64_t>(8, (live + sms - 1) / sms);
    // A warp per item where many have few keys: 320 items of 100, 250 and 500 keys (D 128) 9.7, 16 and 27 us,
    // clusters 12, 17 and 25; 800 items 13, 22 and 38, clusters 21, 29 and 42, of 1000 keys 70 and 71 (of 100
    // to 1000 keys 55 and 46: a warp waits for the longest); D 64 alike.
    const bool by_warp = a.kv_dtype != PA_F32 && live > slots && most <= (per_sm >= 5 ? 768 : 384);
    const int warps = by_warp ? per_sm : 0;
    // Long contexts first where a second wave of CTAs would otherwise end with one: 512 items of 1600
    // to 6404 keys 194 -> 155 us, 800 of 500 to 2500 108 -> 97; past four waves the lengths even out
    // and the ranking only costs (1600 items of 500 to 2500 keys 108 -> 114 us).
    p.by_length = !by_warp && live * cluster > slots && live * cluster <= 4 * slots && a.num_seqs <= kMostRanked;
    if (by_warp) p.unit = a.block_size >= 16 && most >= a.head_dim * per_sm ? 2 : 1;
    if (items * cluster > INT32_MAX) return PA_ERR_INVALID_ARG;
    const dim3 grid((unsigned)(items * cluster));
    const int64_t rows = (int64_t)a.num_blocks * a.block_size;
    CUtensorMap km, vm;
    for (int i = 0; i < 2; ++i) {
        CUtensorMap *m = i ? &vm : &km;
        const void *base = i ? a.value_cache : a.key_cache;
        const int rc = a.kv_dtype == PA_F32
                           ? make_kv_tensor_map(m, base, a.kv_dtype, a.head_dim, a.num_kv_heads, rows, 1, 8 * p.unit)
                           : make_kv_block_map(m, base, a.kv_dtype, a.head_dim, a.num_kv_heads, rows, 8 * p.unit);
        if (rc != PA_OK) return rc;
    }
    switch (a.kv_dtype) {
        case PA_F32:
            return a.head_dim == 64 ? launch_f32<64, true>(p, cluster, grid, columns, km, vm, a.stream)
                                    : launch_f32<128, true>(p, cluster, grid, columns, km, vm, a.stream);
        case PA_F16:
            return a.head_dim == 64 ? launch_16<F16, 64, true>(p, cluster, grid, items, warps, km, vm, a.stream)
                                    : launch_16<F16, 128, true>(p, cluster, grid, items, warps, km, vm, a.stream);
        case PA_BF16:
            return a.head_dim == 64 ? launch_16<BF16, 64, true>(p, cluster, grid, items, warps, km, vm, a.stream)
                                    : launch_16<BF16, 128, true>(p, cluster, grid, items, warps, km, vm, a.stream);
    }
    return PA_ERR_UNSUPPORTED;
}

}  // namespace

int launch_cross(const CrossArgs &c) {
    const PrefillArgs &a = c.a;
    // Every kernel that a call with this type and head dimension may take is loaded by the first one on
    // a device, so that any later one may be captured.
    if (a.kv_dtype == PA_F32) {
        const int rc = a.head_dim == 64 ? load_f32<64, true>() : load_f32<128, true>();
        return rc == PA_OK ? launch_cross_rows(c) : rc;
    }
    const bool half = a.kv_dtype == PA_F16, wide = a.head_dim == 128;
    int rc = half ? (wide ? load_16<F16, 128, true>() : load_16<F16, 64, true>())
                  : (wide ? load_16<BF16, 128, true>() : load_16<BF16, 64, true>());
    if (rc == PA_OK) rc = load_cross_chunk(a.kv_dtype, a.head_dim);
    if (rc != PA_OK) return rc;
    // The rows' kernel has eight columns, the chunks' a tile of 128.  Above eight the keys are streamed once
    // for every eight columns, which is still the faster as long as that fills the chip no more than
    // clusters of eight CTAs do (one sequence of 4000 keys: 32 items 12.6 us, 15.3 on the chunks'
    // kernel; 64 items 20.1 and 16.5).
    const int64_t columns = (int64_t)std::min(a.max_query_len, a.num_tokens) * (a.num_heads / a.num_kv_heads);
    const int64_t items = (int64_t)a.num_seqs * ((columns + 7) / 8) * a.num_kv_heads;
    return columns <= 8 || items * 8 <= 2 * device_sm_count() ? launch_cross_rows(c) : launch_cross_chunk(c);
}

}  // namespace pa
