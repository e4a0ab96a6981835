// Host check of the decode kernels' index arithmetic (built and run by tests/test_decode_abi.py, no
// GPU): what the kernels read from device memory (positions, counts, lengths, sequences, table
// entries) runs through the same functions here, over valid and invalid values, and every result
// has to lie inside the buffers.
#include <climits>
#include <cstdio>
#include <vector>

#include "decode_rows.cuh"

using namespace stem;

static int fail(const char* what, long long a, long long b) {
  std::printf("%s %lld %lld\n", what, a, b);
  return 1;
}

int main() {
  const int nseq = 2, max_blocks = 3, pages = 4;
  for (int block : {64, 128}) {
    const std::vector<int32_t> odd = {INT_MIN, -block, -1,        0,          1,
                                      block - 1, block, block + 1, 3 * block - 1, 3 * block,
                                      3 * block + 1, INT_MAX - 1, INT_MAX};
    std::vector<int32_t> table(nseq * max_blocks, 0);
    KvCache c{};
    c.table = table.data();
    c.num_pages = pages;
    c.Hkv = 2;
    c.block = block;
    c.nseq = nseq;
    c.max_blocks = max_blocks;
    c.record = 4096;
    // pages
    for (int32_t p : odd)
      for (int s = 0; s < nseq; ++s)
        for (int j = 0; j < max_blocks; ++j) {
          table[s * max_blocks + j] = p;
          int32_t status = 0;
          const int got = kv_page(c, s, j, &status);
          const bool in = p >= 0 && p < pages;
          if (got != (in ? p : -1) || status != (in ? 0 : STEM_ERR_ARG)) return fail("page", p, got);
          if (kv_page(c, s, j, nullptr) != got) return fail("page", p, j);
        }
    if (c.at(pages - 1, 1) - c.at(0, 0) != (pages * 2 - 1) * 4096) return fail("at", 0, 0);
    c.record = 65536;
    c.Hkv = 8;
    if (c.at(1 << 20, 7) - c.at(0, 0) != ((1ll << 23) + 7) * 65536) return fail("at", 1, 0);
    // rows of K and V
    const int T = 2 * block;
    for (int32_t pos : odd)
      for (int32_t n : odd) {
        const bool ok = n >= 0 && n <= T && pos >= 0 && 1ll * pos + n <= 3ll * block;
        const int touched = (T + block - 2) / block + 1;  // the launch's grid
        long long rows = 0;
        int32_t status = 0;
        for (int b = 0; b < touched; ++b) {
          int j, first, lo, hi;
          if (!kv_block_rows(c, pos, n, T, b, &status, j, first, lo, hi)) continue;
          if (j < 0 || j >= max_blocks || lo < 0 || hi <= lo || hi > block) return fail("rows", pos, n);
          if (first + lo != rows || first + hi > n) return fail("first", pos, n);
          rows += hi - lo;
        }
        if (rows != (ok ? n : 0)) return fail("count", pos, n);
        if (status != (ok || n == 0 ? 0 : STEM_ERR_ARG)) return fail("status", pos, n);
      }
    // query rows
    for (int32_t seq : odd)
      for (int32_t len : odd)
        for (int mapped = 0; mapped < 2; ++mapped) {
          int32_t status = 0;
          DecodeRows r{};
          r.rows = mapped ? &seq : nullptr;
          r.lens = &len;
          r.status = &status;
          int s, l;
          decode_row(c, r, 0, s, l);
          const int want = mapped ? seq : 0;
          const bool ok = want >= 0 && want < nseq && len >= 0 && len <= 3 * block;
          if (s < 0 || s >= nseq || l != (ok ? len : 0) || (ok && s != want))
            return fail("row", seq, len);
          if (status != (ok ? 0 : STEM_ERR_ARG)) return fail("row status", seq, len);
        }
  }
  // parts of the attention's items: as many as CTAs, however many entries (the totals a call may
  // have end at 2^31 - 1)
  for (int at_once : {296, 444, 592})
    for (int total : {0, 1, 2, 295, 296, 297, 1 << 20, 1431655764, 1431655766, INT_MAX - 1,
                      INT_MAX}) {
      const int chunk = part_entries(total, at_once, 2);
      if (chunk < 2) return fail("chunk", total, chunk);
      for (long long n : {1ll, 2ll, 7ll, 4095ll, 4096ll}) {  // items of n entries, the last has the rest
        const long long items = (total + n - 1) / n;
        const long long last = total - (items - 1) * n;
        const long long parts =
            items == 0 ? 0 : (items - 1) * ((n + chunk - 1) / chunk) + (last + chunk - 1) / chunk;
        if (parts > items + at_once) return fail("parts", total, parts);
      }
    }
  std::printf("ok\n");
  return 0;
}
