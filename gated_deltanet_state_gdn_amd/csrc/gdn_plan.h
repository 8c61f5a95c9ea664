// How the suffix and decode operators cut their work: choices of the host from sizes alone, the same for
// a call and for the query of its workspace.  Plain functions of integers, so that host code can
// include and test them.
#pragma once
#include <stdint.h>

namespace gdn {

// ------------------------------------------------------------- state space scan
constexpr int kScanChunk = 64;      // tokens of a chunk

// Time of a scan whose longest sequence has `longest` chunks, cut into s segments: one launch, or the
// states, their chain and the outputs in three.  In microseconds, fitted; `work` is the chunks of 64
// columns that a CU has.  Alone on its CU a bf16 chunk of d_k = 128 takes 3.6 us in one launch and 4.3 in
// two, 1.5 and 2.0 of it the CU's own for every other workgroup there; fp32, bound by its products, 9.3
// and 11.4 alone and 10.3 and 13.5 of the CU.  Three launches cost 7.5 us more than one, and every
// segment's state is written twice and read twice.
inline double scan_time(int64_t s, int64_t longest, double work, double states, int32_t d_k, int bf16)
{
    const double k = (double)((longest + s - 1) / s);
    const double alone = k * (s == 1 ? (bf16 ? 3.6 : 9.3) : bf16 ? 4.3 : 11.4);
    const double shared = s == 1 ? (bf16 ? k * 2.1 + work * 1.5 : work * 10.3) : bf16 ? k * 2.3 + work * 2.0 : work * 13.5;
    const double moved = (double)(s < longest ? s : longest) * states * d_k * 64 * 4 * 4 / 8e6;
    return (alone > shared ? alone : shared) * (0.5 + d_k / 256.0) + (s == 1 ? 4.0 : 11.5 + moved);
}

// Segments a sequence is cut into: the least time, as the mean of equal sequences and of ragged ones
// whose longest is 3.5 times the mean; one where every CU has two workgroups without.  The host does not
// know the lengths: 3.5 comes from the ragged batches that this was fitted with (lengths by the square of a
// uniform number, one in ten empty: 2.8 to 3.7); others have their answer too, if not in the least time.
// At most four workgroups a CU that are not empty (bf16: what runs at once) or eight (fp32, whose chunks
// are long beside their states).
// One sequence of 32768 tokens, 32 heads: 192 us in 32 segments, 254 in 21, 225 in 64 (all before the outputs'
// second term, which adds 7); 16 of 512 tokens, 8 heads, 34.1 in one launch and 32.7 in four segments; one of
// 512 tokens, 4 heads, 32.5 in one and 15.9 in eight; 16 of 512 with 32 heads 44.7 in one and 69.5 in two;
// fp32, 24 ragged ones of 292 on average, 4 heads of 64: 109 in one, 39.3 in twelve, 42.6 in 21.
inline int32_t scan_segments(int32_t n_seqs, int32_t h_v, int32_t d_k, int32_t d_v, int bf16, int64_t tokens)
{
    if (n_seqs <= 0 || tokens <= kScanChunk) return 1;
    const int64_t chunks = (tokens + kScanChunk - 1) / kScanChunk, mean = (chunks + n_seqs - 1) / n_seqs;
    const int64_t longest = mean * 7 / 2 < chunks ? mean * 7 / 2 : chunks;
    const double chains = (double)n_seqs * h_v * d_v / 64;               // of 64 columns
    if (chains >= 512) return 1;
    const double work = (double)chunks * h_v * d_v / 64 / 256, part = (double)chunks / (double)(n_seqs * longest);
    const double filled = chains * (part < 1.0 ? part : 1.0);            // workgroups a segment that are not empty
    const int64_t places = (int64_t)((bf16 ? 1024 : 2048) / filled), most = places < longest ? places : longest;
    int64_t best = 1;
    double least = 0.0;
    for (int64_t s = 1; s == 1 || s <= most;) {
        const double t = scan_time(s, mean, work, chains, d_k, bf16) + scan_time(s, longest, work, filled, d_k, bf16);
        if (s == 1 || t < least) {
            least = t;
            best = s;
        }
        const int64_t next = s + s / 8 + 1;
        s = s < most && next > most ? most : next;
    }
    return (int32_t)best;
}

// ------------------------------------------------------------- paged attention
struct AttnPlan {
    bool decode;
    int32_t rows;               // rows of a workgroup
    int32_t waves;              // of a workgroup, if decode
    int32_t splits, split_keys; // split s covers keys [s split_keys, (s + 1) split_keys)
};

// Waves of a workgroup: two workgroups' tiles fit the LDS of a CU (rows of 1 KB aside), so that one's
// first loads and last sums overlap with the other's keys; or twice as many waves for a workgroup of its
// own CU, where workgroups are few (rows of 1 KB do not fit twice).
constexpr int decode_waves(int row_bytes) { return row_bytes >= 512 ? 2 : 4; }
constexpr bool decode_wide(int row_bytes) { return row_bytes < 1024; }

// Keys of a split for many bf16 rows: the least of the rounds of workgroups, each as long as its tiles of
// 64 keys (3.7 us for 256 rows of d = 256 and by d) and 3 us of start and end, and the join.  The chip
// holds one workgroup of 256 rows a CU, or two of 128 in as long: 1024 tokens of 8 heads on each of 2 cache
// heads over 32K, 64 workgroups, take 480 us in four splits, 583 in three, 726 in five, 503 in eight.
inline int32_t long_splits(int64_t rows, int64_t tiles, int64_t places, int d, int32_t max_kv)
{
    const int32_t all = max_kv > 0 ? (max_kv + 63) / 64 : 1;
    const double tile = 3.7 * d / 256;
    int32_t best = all;
    double least = 0.0;
    for (int32_t splits = 1; splits == 1 || (2 * splits <= all + 1 && splits <= 64); ++splits) {
        const int32_t k = (all + splits - 1) / splits;
        const double rounds = (double)((tiles * splits + places - 1) / places);
        const double t = rounds * (k * tile + 3.0) + (splits > 1 ? 5.0 + (double)rows * splits * d * 8 / 4e6 : 0.0);
        if (splits > 1 && t >= least) continue;
        least = t;
        best = k;
    }
    return best * 64;
}

// Keys of a split where rows are few and contexts short: the least of what the workgroups' tiles take,
// one after the other and in as many rounds as there are workgroups for three quarters of the places
// (which is where uneven ones began to count), the reads, of half the longest context (of contexts
// spread evenly up to it, the ragged ones that this was fitted with), and the join of more than one
// split.  In microseconds, fitted to times of 6 to 300 sequences of 96 to 4000 keys, equal
// and ragged; d = 128, bf16, 2 cache heads: 20 sequences of 256 keys 6.6 us in one split and 9.3 in two,
// of 1000 keys 13.6 in one and 10.3 in eight; 160 of 500 keys 17.0 in one and 23.0 in three.  Twice the
// waves: 6 sequences of 128 keys, d = 256, 7.2 us for 8.7 with two; of 512, d = 128, 8.2 for 8.9 with four.
inline int32_t short_splits(int64_t rows, int64_t tiles, int64_t heads, int d, int32_t max_kv, int bf16, int waves, double &least)
{
    const int row = d * (bf16 ? 2 : 4);
    const int64_t places = 192 * (waves * 64 * row <= 80 * 1024 ? 2 : 1);
    // a tile: a wave's 32 keys; with eight waves a SIMD has two, which hold each other up
    const double tile = (bf16 ? 0.3 + 0.006 * d : 0.6 + 0.018 * d) * (waves == 8 ? 1.5 : 1.0);
    const double reads = (double)heads * max_kv * row / 5e6;
    const int32_t all = max_kv > 0 ? (max_kv + 32 * waves - 1) / (32 * waves) : 1;    // tiles of a wave
    int32_t best = all;
    least = 0.0;
    for (int32_t splits = 1; splits <= all; ++splits) {
        const int32_t k = (all + splits - 1) / splits;
        const double products = (double)((tiles * splits + places - 1) / places) * (2.0 + k * tile);
        const double join = splits > 1 ? 5.0 + (double)rows * splits * d * 8 / 4e6 : 0.0;
        const double t = products + reads + join;
        if (splits > 1 && t >= least) continue;
        least = t;
        best = k;
    }
    return best * 32 * waves;
}

inline AttnPlan attn_plan(int64_t total, int32_t n_seqs, int32_t h_q, int32_t h_kv, int32_t d, int32_t max_kv, int bf16)
{
    const int64_t G = h_q / h_kv;
    AttnPlan p;
    // fp32 in few workgroups over short contexts too: 16 rows to a workgroup whose waves share the keys
    // (5 prompts of 47 tokens on average, 2 heads of 256, 100 keys: 16.8 us for 21.5 with 64 rows; over
    // 8K keys the reads count, 60 us with 64 rows for 94)
    p.decode = total * G <= 32 * (int64_t)n_seqs || (!bf16 && max_kv <= 512 && (total * G / 64 + n_seqs) * h_kv < 128);
    // bf16: 256 rows share a tile of keys where sequences have them.  fp32 products take sixteen times as
    // long and the reads beside them do not count: 64 rows, and splits for several workgroups a CU, for
    // their even spread.
    // Few rows: 32 to a workgroup read the keys once where 16 would twice (32 ragged sequences of up to
    // 8K keys, 32 query heads on each of 2 cache heads, d = 64: 32.3 us for 40.4; 16 sequences, 24 heads
    // on one, d = 256: 31.3 for 42.2).  At d = 128 the first call takes 67.4 us for 59.2 with 16, and
    // fp32 gains nothing (25.2 for 25.6).
    if (p.decode) p.rows = bf16 && d != 128 && total * G > 16 * (int64_t)n_seqs ? 32 : 16;
    else p.rows = !bf16 ? 64 : total * G >= 192 * (int64_t)n_seqs ? 256 : 128;
    const int64_t tiles = (total * G / p.rows + n_seqs) * h_kv;
    const int row = d * (bf16 ? 2 : 4);
    p.waves = decode_waves(row);
    const int64_t active = total * G / p.rows > n_seqs ? total * G / p.rows : n_seqs;
    if (p.decode && max_kv < 4096) {
        double t, wide;
        p.split_keys = short_splits(total * h_q, active * h_kv, (int64_t)n_seqs * h_kv, d, max_kv, bf16, p.waves, t);
        if (decode_wide(row)) {
            const int32_t keys = short_splits(total * h_q, active * h_kv, (int64_t)n_seqs * h_kv, d, max_kv, bf16, 2 * p.waves, wide);
            if (wide < t) p.waves *= 2, p.split_keys = keys;
        }
    } else if (bf16 && !p.decode) {
        // of a sequence's last tile of rows half is expected to be empty
        const int64_t filled = (total * G + p.rows - 1) / p.rows + (n_seqs - 1) / 2;
        p.split_keys = long_splits(total * h_q, filled * h_kv, 256 * (256 / p.rows), d, max_kv);
    } else if (p.decode) {
        // Long contexts may be ragged, and the longest then runs alone: splits of 1024 keys (40 requests of
        // up to 12000 keys, 8 cache heads of 128: 225 us, 303 in splits of 4000; 64 of up to 16000, 2 of 64:
        // 65 us, 83 and, in splits of 170, 69), of fewer where that makes less than two workgroups a CU,
        // but of four tiles (one token over 8K keys: 14.9 us, 16.3 in splits of 64, 17.5 of 256).  fp32: half
        // of both, whose tiles take twice as long (3 requests of up to 16000, 4 of 128: 19.9 us for 24.9).
        // A loose bound makes at most some 8192 workgroups, most of them empty, and a workspace for as many;
        // where there are as many without splits, none are split.
        const int64_t chains = active * h_kv, all = max_kv * (chains < 8192 ? chains : 8192);
        const int64_t few = all / (bf16 ? 512 : 1024), many = all / 8192;
        const int64_t most = bf16 ? 1024 : 512, keys = many > most ? many : few > most ? most : few;
        p.split_keys = (int32_t)(keys < 128 ? 128 : (keys + 127) / 128 * 128);
        const int64_t blocks = chains * (((int64_t)max_kv + p.split_keys - 1) / p.split_keys);
        if (decode_wide(row) && blocks <= 256 && p.split_keys >= 64 * p.waves) p.waves *= 2;
    } else {
        // fp32: for several workgroups a CU.  No join for a few tiles, else at least 128 keys, over a short
        // context, where a tile takes 4 us, 64 (55 prompts of 11 tokens over 110: 16.1 us, 20.3 of 128).
        const int64_t want = tiles > 0 && tiles < 2048 ? 2048 / tiles : 1, keys = (max_kv + want - 1) / want;
        const int64_t least = max_kv <= 256 ? 256 : max_kv < 4096 ? 64 : 128;
        p.split_keys = (int32_t)((keys > least ? keys + least - 1 : least) / least * least);
    }
    p.splits = max_kv > 0 ? (int32_t)(((int64_t)max_kv + p.split_keys - 1) / p.split_keys) : 1;
    return p;
}

// ------------------------------------------------------------- attention behind shared prefixes
struct SharedPlan {
    AttnPlan prefix, own;       // no splits: the side has no keys
    bool fine;                  // probabilities of 16 bits whatever the form: few rows a sequence, as without groups
};

// The form of few rows for one side of a call whose parts are joined in any case: the keys of a split that take the
// least time, in microseconds.  `units` are groups or sequences, which have all their rows in as many tiles.
// As short_splits, fitted with it: rounds of workgroups and their tiles; the reads from memory; and, where several
// tiles of rows read the same keys, theirs from the caches.  256 rows on each of 2 cache heads of 128, bf16, 12000
// keys, up to 300 own ones: 29.5 us in splits of 1024, 35.2 of 512, 41.4 of 256; 64 rows: 21.8, 19.6, 17.1.
inline double few_rows_side(int64_t total, int64_t units, int32_t h_q, int32_t h_kv, int32_t d, int32_t most, int bf16, int32_t rows,
                            int32_t waves, bool shared, int32_t &keys)
{
    const int row = d * (bf16 ? 2 : 4);
    const int64_t G = h_q / h_kv, filled = (total * G + rows - 1) / rows, tiles = (filled > units ? filled : units) * h_kv;
    const int64_t places = 192 * (waves * 64 * row <= 80 * 1024 ? 2 : 1);
    const double tile = (bf16 ? 0.3 + 0.006 * d : 0.6 + 0.018 * d) * (waves == 8 ? 1.5 : 1.0) * (rows == 32 ? 1.3 : 1.0);
    const double reads = (double)units * h_kv * most * row * (shared ? 2 : 1) / 5e6;           // own keys: half of the longest
    const double caches = shared ? (double)tiles * most * row * 2 / 14e6 : 0.0;
    const int64_t all = most > 0 ? ((int64_t)most + 32 * waves - 1) / (32 * waves) : 1;        // tiles of a wave
    int64_t best = all;
    double least = 0.0;
    for (int64_t splits = 1; splits <= all && splits <= 512; splits += 1 + splits / 16) {
        const int64_t k = (all + splits - 1) / splits;
        const double products = (double)((tiles * splits + places - 1) / places) * (2.0 + (double)k * tile);
        const double t = (products > caches ? products : caches) + reads + (double)total * h_q * (double)splits * d * 8 / 4e6;
        if (splits > 1 && t >= least) continue;
        least = t;
        best = k;
    }
    const int64_t most_keys = (1LL << 30) / (32 * waves) * (32 * waves);
    keys = (int32_t)(best * 32 * waves < most_keys ? best * 32 * waves : most_keys);
    return least;
}

// The sides' forms.  Own keys: as without groups, few rows a sequence or many.  A prefix's rows are those of its group, but
// their form of few rows costs only what it reads from the caches again for every 16 rows, and with the own keys in
// the same form one launch takes both (two requests over 1024 tokens, 2 heads of 256: 14.0 us for 21.3).  bf16: the
// form of many rows where its time, by long_splits' terms and another launch, is less: 512 rows on each of 2 heads of 256
// over 31744 tokens, and up to 1024 own ones, take 97 us for 177; 256 rows over 12288, up to 300, 53.7 for 48.4.  fp32: up to 512 rows for d <= 128 (256 rows
// of 128 over 12000: 66 us for 80), but not for 256, whose rows of 1 KB leave a workgroup two waves (141 for 197).
inline SharedPlan shared_plan(int64_t total, int32_t n_seqs, int32_t n_groups, int32_t h_q, int32_t h_kv, int32_t d,
                              int32_t max_prefix, int32_t max_own, int bf16)
{
    SharedPlan p;
    p.prefix = attn_plan(total, n_groups, h_q, h_kv, d, max_prefix, bf16);
    p.own = attn_plan(total, n_seqs, h_q, h_kv, d, max_own, bf16);
    const int64_t rows = total * (h_q / h_kv);
    p.fine = rows <= 32 * (int64_t)n_seqs;
    const bool own_few = max_own == 0 ? rows <= 32 * (int64_t)n_groups : p.own.decode;
    if (own_few) {
        const int row = d * (bf16 ? 2 : 4), narrow = decode_waves(row);
        const int32_t tile = max_own > 0 ? p.own.rows : p.prefix.decode ? p.prefix.rows : 16;
        double least = 0.0, own_least = 0.0;
        AttnPlan prefix = p.prefix, own = p.own, alone = p.own;    // own: next to the prefix's form of few rows; alone: without
        for (int waves = narrow; waves <= (decode_wide(row) ? 2 * narrow : narrow); waves *= 2) {
            int32_t pk, ok;
            const double pt = max_prefix > 0 ? few_rows_side(total, n_groups, h_q, h_kv, d, max_prefix, bf16, tile, waves, true, pk) : (pk = 32, 0.0);
            const double ot = max_own > 0 ? few_rows_side(total, n_seqs, h_q, h_kv, d, max_own, bf16, tile, waves, false, ok) : (ok = 32, 0.0);
            if (waves == narrow || ot < own_least) {
                own_least = ot;
                alone.waves = waves;
                alone.split_keys = ok;
            }
            if (waves > narrow && pt + ot >= least) continue;
            least = pt + ot;
            prefix.waves = own.waves = waves;
            prefix.split_keys = pk;
            own.split_keys = ok;
        }
        bool few = rows <= 32 * (int64_t)n_groups || (!bf16 && d <= 128 && rows <= 512 * (int64_t)n_groups);
        if (bf16 && !few) {
            int32_t keys;
            const double one = few_rows_side(total, n_groups, h_q, h_kv, d, max_prefix, bf16, tile, prefix.waves, true, keys);
            const int64_t filled = ((rows + p.prefix.rows - 1) / p.prefix.rows + (n_groups - 1) / 2) * h_kv, places = 256 * (256 / p.prefix.rows);
            const double rounds = (double)((filled * p.prefix.splits + places - 1) / places);
            const double many = rounds * (p.prefix.split_keys / 64 * 3.7 * d / 256 + 3.0) + (double)total * h_q * p.prefix.splits * d * 8 / 4e6 + 9.0;
            few = one <= many;
        }
        if (!few) own = alone;
        // contexts of 4096 keys and more may be ragged: splits that do not leave the longest alone
        if (max_own >= 4096 && own.split_keys > p.own.split_keys) own.split_keys = p.own.split_keys;
        p.own.rows = tile;
        p.own.decode = true;
        p.own.waves = own.waves;
        p.own.split_keys = own.split_keys;
        if (few) {
            p.prefix.rows = tile;
            p.prefix.decode = true;
            p.prefix.waves = prefix.waves;
            p.prefix.split_keys = prefix.split_keys;
        }
    }
    p.prefix.splits = max_prefix > 0 ? (int32_t)(((int64_t)max_prefix + p.prefix.split_keys - 1) / p.prefix.split_keys) : 0;
    p.own.splits = max_own > 0 ? (int32_t)(((int64_t)max_own + p.own.split_keys - 1) / p.own.split_keys) : 0;
    return p;
}

// ------------------------------------------------------------- next token
constexpr int kSampleBins = 256;

// Elements of a chunk, one workgroup's.  Small ones are read by more workgroups, sooner; a row's many of them take its
// workgroup longer to join, and all of them more to write.  bf16, 2048 against 8192: one row of 32768 takes 19.8 us and 21.3,
// of 100000 22.8 and 21.6; 48 rows of 50000 36.5 and 36.8, 100 rows 39.5 and 38.0; 32 rows of 262144 62 and 51.
// So many rows have small ones, of up to 65536 elements: those of fewer than 400 large ones.
inline int64_t sample_small_rows(int32_t vocab) { return vocab <= 65536 ? 399 / ((vocab + 8191) / 8192) : 0; }
inline int32_t sample_chunk(int64_t rows, int32_t vocab) { return rows <= sample_small_rows(vocab) ? 2048 : 8192; }

}  // namespace gdn
