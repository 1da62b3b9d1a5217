// decode_window.cu -- decode attention over a sliding window with sinks (kernels: stream_rows.cuh).
#include "stream_rows.cuh"

namespace pa {

int launch_decode_window(const DecodeArgs &a) {
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
    p.window = a.window;
    p.num_sinks = a.num_sinks;
    p.qk_scale_log2 = a.scale * kLog2e;
    p.status = a.status;
    const int64_t rows = (int64_t)a.num_blocks * a.block_size;
    if (rows <= 0 || rows > INT32_MAX) return PA_ERR_INVALID_ARG;
    // The cluster size: the CTAs of one full wave, but none with less than one stage of keys
    // (two past eight CTAs).  A CTA past the first wave costs more than its shorter run of keys
    // gives back, and clusters start slowly: 256 (sequence, kv head) pairs of 1028 keys took 23,
    // 29, 40 and 61 us in clusters of 1, 2, 4 and 8; 61 pairs of 790 keys 11.8, 8.6, 7.0 and
    // 11.0 us; 8 pairs of 516 keys 11.1, 8.2, 6.5, 5.4 and (16) 5.7 us, of 4100 keys (8) 9.5 and
    // (16) 7.7 us (bf16).
    const int sms = std::max(1, device_sm_count());
    const int64_t slots = 2 * sms;  // resident CTAs
    const int64_t most = std::min<int64_t>(a.max_context_len, (int64_t)a.window + a.num_sinks);  // keys of a row
    const int64_t stage_keys = 16384 / (a.head_dim * (a.kv_dtype == PA_F32 ? 4 : 2));
    const int64_t pairs = (int64_t)a.num_seqs * a.num_kv_heads;
    // What is resident in clusters of a size, as the parts of the chip do not divide evenly: of
    // 304 CTAs 296 in fours, 288 in eights, 224 in sixteens.  One cluster more is a second wave
    // (76 pairs of 333 fp32 keys 6.0 us in twos, 9.1 in fours; 16 pairs of 2004 keys 7.4 in eights,
    // 11.6 in sixteens).
    auto fit = [&](int size) { return slots * (size <= 2 ? 64 : size == 4 ? 63 : size == 8 ? 61 : 48) / 64; };
    int cluster = 1;
    while (cluster < 16 && pairs * cluster * 2 <= fit(cluster * 2) &&
           most > stage_keys * cluster * (cluster < 8 ? 1 : 2))
        cluster *= 2;
    // A second wave that few pairs start takes as long as the first: two CTAs per pair halve it (312
    // to 384 pairs of 4096 keys 136 to 141 -> 122 to 128 us; 448 pairs are equal, of 2048 keys 77 ->
    // 82).
    if (pairs > slots && pairs <= slots * 4 / 3 && most >= 16 * stage_keys) cluster = 2;
    // A box of a whole block where one warp's issue of the boxes bounds a CTA (about 70 clocks
    // each: 8 pairs of 4100 keys 9.0 -> 7.7 us) or where the rows past the borders that it brings
    // along are few (1024 pairs of 4112 keys in blocks of 16, 333 -> 318 us; but 256 pairs of 1028
    // keys in blocks of 32, 23.3 -> 24.0 us).
    p.unit = cluster > 1 || most >= 64 * (int64_t)a.block_size ? a.block_size / 8 : 1;
    // A warp per pair where the clusters would be single CTAs in more than one wave, of rows of
    // about a thousand keys at most: 1024 pairs of 132, 516 and 1028 keys 29.8 -> 16.4, 59.7 -> 47.3
    // and 95.5 -> 87.7 us, 320 pairs of 516 keys 27.2 -> 24.6 us.  Of 2052 keys the two are equal,
    // of 4112 the clusters faster (318 and 332 us), and rows of unequal length leave the longest
    // to one warp: contexts of 10 to 1000 keys 52.6 -> 50.8, of 10 to 2000 90.8 -> 99 us.  Boxes of
    // 16 keys where the rows are long for the warps on an SM (320 pairs of 516 keys 26.3 -> 24.6,
    // but 1024 pairs of 132 keys 16.4 -> 17.9 us).
    // A step of 16 keys takes a warp 0.6 us at least, so at head dimension 64 (half the bytes) a few
    // warps per SM fall behind: 400 pairs of 260 keys 13.5 and 14.0 us (clusters), of 1004 keys 40.3
    // and 31.4; 800 pairs 44.3 and 47.1.
    const int per_sm = (int)std::min<int64_t>(8, (pairs + sms - 1) / sms);
    const bool by_warp = a.kv_dtype != PA_F32 && pairs > slots && pairs <= INT32_MAX &&
                         most <= (per_sm * a.head_dim >= 320 ? 1152 : 384);
    const int warps = by_warp ? per_sm : 0;
    if (by_warp) p.unit = a.block_size >= 16 && most >= a.head_dim * per_sm ? 2 : 1;
    const dim3 grid(cluster, a.num_kv_heads, a.num_seqs);
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
            return a.head_dim == 64 ? launch_f32<64, false>(p, cluster, grid, p.group, km, vm, a.stream)
                                    : launch_f32<128, false>(p, cluster, grid, p.group, km, vm, a.stream);
        case PA_F16:
            return a.head_dim == 64 ? launch_16<F16, 64, false>(p, cluster, grid, pairs, warps, km, vm, a.stream)
                                    : launch_16<F16, 128, false>(p, cluster, grid, pairs, warps, km, vm, a.stream);
        case PA_BF16:
            return a.head_dim == 64 ? launch_16<BF16, 64, false>(p, cluster, grid, pairs, warps, km, vm, a.stream)
                                    : launch_16<BF16, 128, false>(p, cluster, grid, pairs, warps, km, vm, a.stream);
    }
    return PA_ERR_UNSUPPORTED;
}

}  // namespace pa
