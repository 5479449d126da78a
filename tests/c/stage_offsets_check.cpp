/* Walks every load of a stage that the 8-bit product's tiles make, for every
 * number of valid rows, and checks that it reads 16 bytes of its own row inside
 * the panel; a row past the last one has to read the last one.  The panel is
 * (rows - 1) * ld + K bytes, all that an operand's allocation has to hold. */
#include <cstdio>

#include "echo_stage.hpp"

int main()
{
    struct Tile { uint32_t rows, waves; };
    /* rows of x or of w of a tile, waves of its block */
    const Tile tiles[] = {{256, 8}, {128, 8}, {64, 4}, {128, 4}, {64, 2}, {32, 2}};
    struct Row { uint64_t ld, K; };
    const Row lens[] = {{128, 128}, {384, 300}, {4096, 4096}, {131072, 131071}, {(1u << 22) - 16, 1000}};
    unsigned long long loads = 0, wrong = 0, base_past_end = 0;
    for (const Tile& t : tiles)
        for (uint32_t rows = 1; rows <= t.rows; ++rows)
            for (const Row& l : lens) {
                const uint64_t bytes = (rows - 1) * l.ld + l.K;
                const uint64_t k0 = (l.K / 128 - 1) * 128;               /* the last whole stage */
                for (uint32_t j = 0; j < t.rows / (8 * t.waves); ++j) {
                    base_past_end += k0 + 8ull * t.waves * j * l.ld > bytes;
                    for (uint32_t tid = 0; tid < 64 * t.waves; ++tid) {
                        const uint32_t lrow = tid / 64 * 8 + (tid & 63u) / 8, row = lrow + 8 * t.waves * j;
                        const uint32_t chunk = (tid & 7u) ^ echo::i8_key(lrow);
                        const uint64_t at = k0 + echo::stage_offset(row, rows, (uint32_t)l.ld, chunk);
                        const uint64_t own = row < rows ? row : rows - 1;
                        ++loads;
                        wrong += at != own * l.ld + k0 + 16 * chunk || at + 16 > bytes;
                    }
                }
            }
    /* base_past_end: loads whose first row alone is past the panel's end, which a
     * scalar offset that holds that row would leave to the range check */
    std::printf("loads=%llu wrong=%llu base_past_end=%llu\n", loads, wrong, base_past_end);
    return wrong != 0;
}
